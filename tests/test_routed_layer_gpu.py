"""The routing, int8 product and combine calls where offsets pass 32 bits, where two
captured graphs share a workspace, next to guard bytes, and together as one layer that is
captured and replayed."""

import math

import numpy as np
import pytest
import torch

import _routed_reference as ref
import mixture_experts_ffn_14_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def test_route_offsets_past_32_bits():
    T, E, k = 2_100_001, 1024, 3                       # 2.15e9 logits
    l = torch.empty((T, E), dtype=torch.bfloat16, device=DEV)
    for a in range(0, T, 100_000):
        l[a:a + 100_000].normal_(generator=gen(a))
    r = moe.moe_topk_route(l, k, renormalize=True)
    rows = torch.tensor([0, 31, 32, T // 2, 2_097_151, 2_097_152, 2_097_153, T - 1], device=DEV)
    want = ref.route(l[rows].double().cpu().numpy(), k, renorm=True)
    assert (r["idx"][rows].cpu().numpy() == want["idx"]).all()
    counts = torch.bincount(r["idx"].reshape(-1).long(), minlength=E)
    assert torch.equal(counts, r["counts"].long()) and int(r["offsets"][-1]) == T * k
    flat = r["slot_pos"].reshape(-1).long()
    assert torch.equal(torch.sort(flat).values, torch.arange(T * k, device=DEV))
    assert torch.equal(r["perm_token"][flat].long(), torch.arange(T * k, device=DEV) // k)
    experts = r["idx"].reshape(-1)[torch.argsort(flat)].long()
    assert bool((experts[1:] >= experts[:-1]).all())
    same = experts[1:] == experts[:-1]
    assert bool((r["perm_token"][1:][same] > r["perm_token"][:-1][same]).all())
    g = moe.moe_topk_route_backward(l, r["idx"], r["weights"], renormalize=True)
    got = g[rows].double().cpu().numpy()
    back = ref.route_backward(l[rows].double().cpu().numpy(), want["idx"], r["weights"][rows].double().cpu().numpy(),
                              "softmax", True, 1.0)
    # terms p (g - mean) of at most 1: fp32 roundings of share (26 u for k = 3 logits within 3 of
    # one another), product and mean, then the type's
    assert (np.abs(got - back) <= 120 * U + 2.0 ** -8 * np.abs(back)).all()


def test_combine_offsets_past_32_bits():
    d, k, T = 4096, 2, 5
    R = (1 << 31) // d + 50
    y = torch.empty((R, d), dtype=torch.bfloat16, device=DEV)
    y.fill_(float("nan"))
    rows = torch.tensor([[0, R - 1], [R - 2, 1], [R - 30, -1], [(1 << 31) // d, (1 << 31) // d - 1], [-1, -1]],
                        dtype=torch.int32, device=DEV)
    for r in rows.reshape(-1).tolist():
        if r >= 0:
            y[r] = torch.randn(d, generator=gen(r), device=DEV).to(torch.bfloat16)
    got = moe.moe_combine_topk(y, rows, out_dtype=torch.float32)
    want = sum(torch.where(rows[:, j:j + 1] >= 0, y[rows[:, j].clamp(min=0).long()].float(), 0.0) for j in range(k))
    assert torch.equal(got, want)                      # one addition, rounded once


@pytest.mark.parametrize("R,K,N,n", [(70_000, 64, 32768, 3), (40, 4096, 65536, 9)])
def test_product_offsets_past_32_bits(R, K, N, n):
    # R * N = 2.29e9 outputs; n * K * N = 2.4e9 weights
    rows = [R // n] * (n - 1)
    rows.append(R - sum(rows))
    x = torch.randn((R, K), generator=gen(1), device=DEV).to(torch.bfloat16)
    w = torch.empty((n, K, N), dtype=torch.int8, device=DEV)
    for e in range(n):
        w[e].random_(-127, 128, generator=gen(e))
    s = ((torch.rand((n, N), generator=gen(2), device=DEV) + 0.5) / (127 * math.sqrt(K))).to(torch.bfloat16)
    counts = torch.tensor(rows, dtype=torch.int32, device=DEV)
    out = moe.moe_int8_product(x, w, s, counts=counts)
    ends = np.cumsum(rows)
    for r in sorted({0, 1, R // 2, R - 300 if R > 300 else 3, R - 2, R - 1, (1 << 31) // N + 1 if R > (1 << 31) // N + 1 else 5}):
        e = int(np.searchsorted(ends, r, side="right"))
        xr = x[r].double()
        q = torch.round(127 * xr / xr.abs().max())
        a = float((xr.abs().max() / 127).float())
        want = (q @ w[e].double()) * a * s[e].double()
        err = (out[r].double() - want).abs()
        assert bool((err <= want.abs() * (4 * U + 2.0 ** -8)).all()), r


def layer(E, k, d, f, T, seed):
    g = gen(seed)
    i8 = lambda *s: torch.randint(-127, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    sc = lambda m, fan: ((torch.rand((E, m), generator=g, device=DEV) + 0.5) / (127 * math.sqrt(fan))).to(torch.bfloat16)  # noqa: E731
    w = {"wg": i8(E, d, f), "wu": i8(E, d, f), "wd": i8(E, f, d), "sg": sc(f, d), "su": sc(f, d), "sd": sc(d, f)}

    def run(x, logits, nt, ws=None):
        r = moe.moe_topk_route(logits, k, score=moe.MOE_SCORE_SIGMOID, renormalize=True, n_tokens=nt)
        kw = {} if ws is None else {"workspace": ws}
        h = moe.moe_int8_product(x, w["wg"], w["sg"], index=r["perm_token"], counts=r["counts"], w_up=w["wu"],
                                 s_up=w["su"], **kw)
        y = moe.moe_int8_product(h, w["wd"], w["sd"], counts=r["counts"], gate=r["gate_perm"],
                                 out_dtype=torch.float32, **kw)
        return moe.moe_combine_topk(y, r["slot_pos"], residual=x)

    return run


@pytest.mark.parametrize("T", [3, 64, 700])
def test_captured_layers_that_share_a_workspace(T):
    E, k, d, f = 12, 3, 256, 384
    run = layer(E, k, d, f, T, 5)
    size = max(moe.moe_int8_workspace_size(T * k, d, f, E, with_up=True), moe.moe_int8_workspace_size(T * k, f, d, E))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    graphs, states = [], []
    for i in range(2):
        x = torch.zeros((T, d), dtype=torch.bfloat16, device=DEV)
        logits = torch.zeros((T, E), device=DEV)
        nt = torch.tensor([T], dtype=torch.int32, device=DEV)
        run(x, logits, nt, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(x, logits, nt, ws)
        graphs.append(graph)
        states.append((x, logits, nt, out))
    for step in range(4):
        for i in (0, 1):
            x, logits, nt, _ = states[i]
            x.copy_(torch.randn((T, d), generator=gen(10 * step + i), device=DEV))
            logits.copy_(torch.randn((T, E), generator=gen(100 * step + i), device=DEV))
            nt.fill_(max(0, T - step * (i + 1)))
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        for x, logits, nt, out in states:
            assert torch.equal(out, run(x, logits, nt))          # bit for bit the eager layer's
            assert torch.equal(out[int(nt):], x[int(nt):])       # padding: the residual alone
    assert moe.moe_device_status(ws) == (0, 0)


def test_two_layers_at_once_on_two_streams():
    runs = [layer(8, 2, 512, 640, 0, 1), layer(16, 4, 256, 384, 0, 2)]
    ins = [(torch.randn((T, d), generator=gen(T), device=DEV).to(torch.bfloat16),
            torch.randn((T, E), generator=gen(E), device=DEV)) for T, d, E in ((150, 512, 8), (400, 256, 16))]
    want = [run(x, l, None) for run, (x, l) in zip(runs, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(15):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(runs[i](*ins[i], None))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_nothing_is_written_outside_the_outputs():
    """Outputs and workspaces between guard bytes."""
    def guarded(shape, dtype):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device=DEV)
        return buf, buf[1024:1024 + n].view(dtype).view(shape)

    def intact(bufs):
        return all(bool((b[:1024] == 0xA5).all()) and bool((b[-1024:] == 0xA5).all()) for b in bufs)

    for T, E, k in ((1, 8, 2), (77, 33, 3), (300, 60, 6)):
        l = torch.randn((T, E), generator=gen(T), device=DEV)
        shapes = {"idx": ((T, k), torch.int32), "weights": ((T, k), torch.float32), "scores": ((T, E), torch.float32),
                  "counts": ((E,), torch.int32), "offsets": ((E + 1,), torch.int32), "perm_token": ((T * k,), torch.int32),
                  "perm_slot": ((T * k,), torch.int32), "slot_pos": ((T, k), torch.int32), "gate_perm": ((T * k,), torch.float32)}
        both = {n: guarded(*s) for n, s in shapes.items()}
        wsb, ws = guarded((moe.moe_topk_workspace_size(T, E, k),), torch.uint8)
        moe.moe_topk_route(l, k, want_scores=True, out={n: t for n, (_, t) in both.items()}, workspace=ws)
        gb, g = guarded((T, E), torch.float32)
        moe.moe_topk_route_backward(l, both["idx"][1], both["weights"][1], out=g)
        torch.cuda.synchronize()
        assert intact([b for b, _ in both.values()] + [wsb, gb])
    for R, K, N, n in ((1, 16, 16, 1), (37, 144, 272, 4), (130, 1040, 400, 2), (900, 272, 336, 3)):
        rows = [R // n] * n
        x = torch.randn((R, K), generator=gen(R), device=DEV)
        w = torch.randint(-127, 128, (n, K, N), generator=gen(K), device=DEV, dtype=torch.int8)
        s = torch.ones((n, N), dtype=torch.bfloat16, device=DEV)
        for dtype in (torch.float32, torch.bfloat16):
            for up in (None, w):
                ob, out = guarded((R, N), dtype)
                wsb, ws = guarded((moe.moe_int8_workspace_size(R, K, N, n, moe.MOE_F32, up is not None),), torch.uint8)
                moe.moe_int8_product(x, w, s, counts=torch.tensor(rows, dtype=torch.int32, device=DEV), w_up=up,
                                     s_up=None if up is None else s, out=out, workspace=ws)
                torch.cuda.synchronize()
                assert intact([ob, wsb])
    ob, out = guarded((7, 72), torch.bfloat16)
    moe.moe_combine_topk(torch.ones((14, 72), device=DEV), torch.zeros((7, 2), dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    assert intact([ob])


def test_stream_given_as_a_handle():
    # the handle's own stream is current during the call, 0 being the default stream
    from mixture_experts_ffn_14_b200 import routed

    x = torch.zeros((2, 8), device=DEV)
    mine = torch.cuda.Stream()
    handles = [0, mine.cuda_stream]
    assert torch.cuda.default_stream().cuda_stream == 0
    for other in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(other):
            for h in handles:
                assert routed._on(h, x, lambda: torch.cuda.current_stream().cuda_stream, ()) == h
            assert torch.cuda.current_stream() == other
    # work that is queued on the default stream comes before the call's
    n = 1 << 24
    big = torch.zeros(n, device=DEV)
    logits = torch.zeros((64, 8), device=DEV)
    mine.wait_stream(torch.cuda.default_stream())
    for _ in range(50):
        big.add_(1.0)
    logits[:, 5] = big[n - 64:] / 25                  # 2.0 once all additions are done
    with torch.cuda.stream(mine):
        r = moe.moe_topk_route(logits, 1, stream=0)
    torch.cuda.synchronize()
    assert bool((r["idx"] == 5).all())


def test_given_outputs_count_as_changed_in_place():
    T, E, k, d = 40, 16, 2, 64
    l, y = torch.randn((T, E), device=DEV), torch.randn((T * k, d), device=DEV)
    w, s = torch.ones((1, d, 32), dtype=torch.int8, device=DEV), torch.ones((1, 32), dtype=torch.bfloat16, device=DEV)
    outs = {n: torch.zeros_like(t) for n, t in moe.moe_topk_route(l, k, want_scores=True).items()}
    idx, gw = outs["idx"], torch.zeros((T, k), device=DEV)
    grad, comb, prod = torch.zeros_like(l), torch.zeros((T, d), device=DEV), torch.zeros((T * k, 32), device=DEV)
    calls = [(list(outs.values()), lambda: moe.moe_topk_route(l, k, want_scores=True, out=outs)),
             ([grad], lambda: moe.moe_topk_route_backward(l, idx, gw, out=grad)),
             ([comb], lambda: moe.moe_combine_topk(y, outs["slot_pos"], out=comb)),
             ([prod], lambda: moe.moe_int8_product(y, w, s, out=prod))]
    for given, run in calls:
        before, same = [t._version for t in given], [t._version for t in (l, y, gw, w, s)]
        run()
        assert all(t._version > v for t, v in zip(given, before))
        assert same == [t._version for t in (l, y, gw, w, s)]
    # a value that autograd has kept is not read once it is overwritten
    p = torch.ones((T, d), device=DEV, requires_grad=True)
    loss = (p * comb).sum()
    moe.moe_combine_topk(y, outs["slot_pos"], out=comb)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():                       # tensors without a version
        kept = torch.zeros((T, d), device=DEV)
        assert torch.equal(moe.moe_combine_topk(y, outs["slot_pos"], out=kept), comb)


def test_results_are_no_part_of_an_autograd_graph():
    l = torch.randn((8, 16), device=DEV, requires_grad=True)
    r = moe.moe_topk_route(l, 2, want_scores=True)
    assert not any(t.requires_grad for t in r.values())
    assert not moe.moe_topk_route_backward(l, r["idx"], torch.ones((8, 2), device=DEV)).requires_grad
