"""moe_topk_route, its backward pass and moe_combine_topk on the GPU against 64-bit
references: choices and dispatch exactly, numbers to bounds counted in fp32
roundings (u = 2^-24) of the formula, plus the rounding of the output's type."""

import numpy as np
import pytest
import torch

import _routed_reference as ref
import mixture_experts_ffn_14_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
SCORE = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}
RULE = {"max": moe.MOE_GROUP_MAX, "top2": moe.MOE_GROUP_TOP2_SUM}
INTS = ("idx", "counts", "offsets", "perm_token", "perm_slot", "slot_pos")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def logits_of(T, E, dtype, seed, masked=0.0, std=1.5):
    g = gen(seed)
    l = torch.randn((T, E), generator=g, device=DEV) * std
    if masked:
        l[torch.rand((T, E), generator=g, device=DEV) < masked] = -float("inf")
        l[torch.rand(T, generator=g, device=DEV) < 0.1] = -float("inf")     # rows with nothing left
        l[torch.rand((T, E), generator=g, device=DEV) < 0.05] = float("nan")
    return l.to(dtype)


def spread(l, idx):
    """Largest difference of a row's chosen logits, capped where exp underflows."""
    has = (idx >= 0) & (idx < l.shape[1])
    a = np.take_along_axis(l, np.where(has, idx, 0), 1)
    hi = np.where(has & np.isfinite(a), a, -np.inf).max(1)
    lo = np.where(has & np.isfinite(a), a, np.inf).min(1)
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(hi) & np.isfinite(lo), hi - lo, 0)
    return np.minimum(d, 110)[:, None]


def weight_bound(l, r, kind, renorm):
    """Relative error of a weight, in u. Sigmoid: expf 2, sum 1, quotient 1, scale 1.
    Softmax: expf 2, its argument's rounding, 37 for the sum of 1024 terms, quotient 1,
    scale 1. Renormalised: both of the above on the k shares instead, whose sum has 5
    levels, numerator and denominator alike."""
    if renorm:
        return (20 + 2 * spread(l, r["idx"])) * U
    if kind == "sigmoid":
        return np.full((l.shape[0], 1), 8 * U)
    top = np.where(np.isfinite(l), l, -np.inf).max(1, keepdims=True)
    low = np.where(np.isfinite(l), l, np.inf).min(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return (50 + np.nan_to_num(np.minimum(np.abs(top - low), 110))) * U


def run_and_check(logits, k, kind, bias=None, groups=1, keep=1, rule="max", renorm=False, scale=1.0, n=None,
                  want_scores=False, n_tokens=None, **kw):
    got = moe.moe_topk_route(logits, k, score=SCORE[kind], bias=bias, n_groups=groups, topk_groups=keep,
                             group_rule=RULE[rule], renormalize=renorm, scale=scale, want_scores=want_scores,
                             n_tokens=n_tokens, **kw)
    torch.cuda.synchronize()
    check(got, logits, k, kind, bias, groups, keep, rule, renorm, scale, n)
    return got


def check(got, logits, k, kind, bias=None, groups=1, keep=1, rule="max", renorm=False, scale=1.0, n=None):
    l = logits.double().cpu().numpy()
    r = ref.route(l, k, kind, None if bias is None else bias.double().cpu().numpy(), groups, keep, rule, renorm,
                  scale, n)
    for name in INTS:
        if name in got:
            a = got[name].cpu().numpy()
            assert (a == r[name]).all(), (name, np.argwhere(a != r[name])[:5])
    bound = weight_bound(l, r, kind, renorm)
    w = got["weights"].double().cpu().numpy()
    assert (np.abs(w - r["weights"]) <= bound * np.abs(r["weights"]) + 1e-37).all()
    if "gate_perm" in got:
        assert torch.equal(got["gate_perm"].cpu(), torch.from_numpy(ref.dispatch(r["idx"], w, l.shape[1])["gate_perm"]).float())
    if "scores" in got:
        s = got["scores"].double().cpu().numpy()
        assert (np.abs(s - r["scores"]) <= weight_bound(l, r, kind, False) * r["scores"] + 1e-37).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (31, 2, 2), (32, 8, 1), (33, 33, 5), (64, 60, 6), (65, 64, 8), (100, 96, 4), (257, 160, 6),
    (40, 256, 8), (70, 500, 9), (35, 512, 10), (50, 1000, 32), (33, 1024, 32), (2100, 16, 2)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_sizes(T, E, k, kind, dtype):
    l = logits_of(T, E, dtype, 1000 + T + E)
    bias = torch.randn(E, generator=gen(E), device=DEV) * 0.1
    run_and_check(l, k, kind, want_scores=True)
    run_and_check(l, k, kind, bias=bias, renorm=True, scale=2.5)


@pytest.mark.parametrize("E,groups,keep", [(8, 2, 1), (8, 8, 3), (64, 4, 2), (60, 4, 2), (96, 3, 2), (160, 8, 3),
                                           (256, 8, 4), (256, 32, 5), (512, 16, 16), (1000, 10, 4), (1024, 2, 1)])
@pytest.mark.parametrize("rule", ["max", "top2"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_groups(E, groups, keep, rule, with_bias, kind):
    k = min(8, max(1, E // groups * keep - 1))
    bias = torch.randn(E, generator=gen(E), device=DEV) * 0.1 if with_bias else None
    l = logits_of(70, E, torch.bfloat16, E + groups, masked=0.2)
    run_and_check(l, k, kind, bias=bias, groups=groups, keep=keep, rule=rule, renorm=True)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(8, 3), (96, 16), (256, 8)])
def test_route_masked_rows_and_odd_values(kind, renorm, E, k):
    l = logits_of(90, E, torch.float32, E + k, masked=0.5)
    l[5] = torch.finfo(torch.float32).min          # the type's lowest value everywhere
    l[6] = float("inf")                            # all the largest
    l[7, :] = -float("inf")
    l[7, E // 2] = 1.0                             # one expert left
    l[8] = 0.0
    l[9, ::2] = -0.0                               # equal values of either sign of zero
    l[9, 1::2] = 0.0
    l[10] = -200.0                                 # scores below the fp32 range
    l[11] = 200.0
    l[12] = torch.arange(E, device=DEV) * -30.0
    for bias in (None, torch.zeros(E, device=DEV), torch.randn(E, generator=gen(3), device=DEV)):
        run_and_check(l, k, kind, bias=bias, renorm=renorm, want_scores=True)
    bias = torch.randn(E, generator=gen(4), device=DEV)
    bias[0], bias[1], bias[2] = float("nan"), -float("inf"), float("inf")
    run_and_check(l, k, kind, bias=bias, renorm=renorm)
    if E % 8 == 0:
        run_and_check(l, k, kind, bias=bias, renorm=renorm, groups=8, keep=3, rule="max")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_ties_and_near_ties_go_by_64_bits(kind, dtype):
    # Few distinct logits: ties everywhere, decided by the lower expert.
    E, k = 128, 8
    l = torch.randint(-2, 3, (100, E), generator=gen(8), device=DEV).to(dtype)
    run_and_check(l, k, kind)
    run_and_check(l, k, kind, bias=torch.zeros(E, device=DEV), groups=8, keep=2, rule="top2")
    # score + bias equal up to the rounding of the bias: fp32 cannot order them
    row = (torch.randn(E, generator=gen(9), device=DEV)).to(dtype)
    _, _, s = ref.scores(row.double().cpu().numpy()[None], kind)
    bias = torch.from_numpy((1.0 - s[0]).astype(np.float32)).to(DEV)
    l = row.repeat(40, 1)
    run_and_check(l, k, kind, bias=bias)
    run_and_check(l, k, kind, bias=bias, groups=16, keep=5, rule="top2")
    run_and_check(l, k, kind, bias=bias, groups=16, keep=5, rule="max", renorm=True)


@pytest.mark.parametrize("E", [33, 64, 96, 128, 256, 512, 1000])
@pytest.mark.parametrize("span", [3, 40, 3000, 1 << 24])
def test_route_logits_below_the_normal_range(E, span):
    # multiples of 2^-149 of either sign, and at the largest span normal numbers beside them: there a
    # key's lost bits are steps of a fixed size
    steps = torch.randint(-span, span + 1, (60, E), generator=gen(E + span), device=DEV, dtype=torch.int32)
    l = torch.where(steps < 0, -1.0, 1.0) * steps.abs().view(torch.float32)
    assert torch.equal((l.double() * 2.0 ** 149).abs()[steps.abs() < 1 << 23].long(), steps.abs()[steps.abs() < 1 << 23].long())
    l[0] = -1.0
    l[0, 0], l[0, 1] = 2.0 ** -148, 2.0 ** -148 + 2.0 ** -149
    run_and_check(l, 1, "softmax")
    run_and_check(l, 8, "sigmoid", renorm=True)
    for groups in (2, 8, 3):
        if E % groups == 0:
            run_and_check(l, 4, "softmax", groups=groups, keep=1, rule="max")
            run_and_check(l, 4, "softmax", groups=groups, keep=groups - 1, rule="max")
            run_and_check(l, 4, "sigmoid", groups=groups, keep=groups - 1, rule="top2")


@pytest.mark.parametrize("mean", [-100.0, -80.0, -60.0, -40.0, 0.0, 60.0])
@pytest.mark.parametrize("E,k", [(3, 3), (24, 24), (256, 8)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_shares_of_scores_far_below_the_largest(mean, E, k, kind):
    # chosen scores out to e^-60 of the largest, on either side of the fp32 range
    l = mean + 15.0 * torch.randn((64, E), generator=gen(E), device=DEV)
    run_and_check(l, k, kind, renorm=True)
    run_and_check(l, k, kind, renorm=True, bias=torch.randn(E, generator=gen(3), device=DEV))
    idx = moe.moe_topk_route(l, k, score=SCORE[kind], dispatch=False)["idx"]
    gw = torch.randn((64, k), generator=gen(4), device=DEV)
    got = moe.moe_topk_route_backward(l, idx, gw, score=SCORE[kind], renormalize=True)
    a = (l.double().cpu().numpy(), idx.cpu().numpy(), gw.double().cpu().numpy(), kind, True, 1.0)
    assert (np.abs(got.double().cpu().numpy() - ref.route_backward(*a)) <= grad_bound(*a, None, 64)).all()


@pytest.mark.parametrize("E,groups", [(64, 8), (224, 7), (256, 8), (512, 16), (1000, 10), (96, 3)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_infinite_biases_beside_a_near_tie_of_groups(E, groups, kind):
    # the groups at the limit are equal in 32 bits, those far above it hold a bias of +inf
    l = 1.0 + torch.randint(-3, 4, (64, E), generator=gen(E), device=DEV) * 2.0 ** -23
    l[torch.rand((64, E), generator=gen(E + 1), device=DEV) < 0.5] = float("nan")
    bias = torch.randint(-1, 2, (E,), generator=gen(E + 2), device=DEV).float()
    for g in range(0, groups, 3):
        bias[g * (E // groups) + 1:(g + 1) * (E // groups):2] = float("inf")
    bias[E // 2] = -float("inf")
    for keep in range(1, groups):
        for rule in ("max", "top2"):
            run_and_check(l, 5, kind, bias=bias, groups=groups, keep=keep, rule=rule, renorm=True)


@pytest.mark.parametrize("E,groups", [(16, 4), (96, 8), (96, 3), (256, 8), (1000, 10)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_groups_whose_sum_of_two_leaves_the_fp32_range(E, groups, kind):
    # biases of the type's lowest and largest value: a group that sums to -2^129 is still above
    # one that has no expert left
    l = torch.randn((12 * groups, E), generator=gen(E), device=DEV)
    size = E // groups
    low, top = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    for t in range(l.shape[0]):
        g = t % groups
        l[t, :g * size] = -float("inf")              # the first groups have nothing left
        if t >= 6 * groups:
            l[t, (groups - 1) * size:] = -float("inf")
    mixed = torch.where(torch.arange(E, device=DEV) % 3 == 0, low, 0.0)
    ends = torch.where(torch.arange(E, device=DEV) % 5 == 0, top, low)
    for bias in (torch.full((E,), low, device=DEV), torch.full((E,), top, device=DEV), mixed, ends, ends * 0.6):
        for keep in (1, groups - 1):
            run_and_check(l, 2, kind, bias=bias, groups=groups, keep=keep, rule="top2")
            run_and_check(l, 2, kind, bias=bias, groups=groups, keep=keep, rule="max")


@pytest.mark.parametrize("n", [0, 1, 37, 64, 100, 500, -3])
@pytest.mark.parametrize("T", [20, 100])
def test_route_padded_batch(T, n):
    l = logits_of(T, 64, torch.bfloat16, 5)
    l[max(0, min(n, T)):] = float("nan")           # whatever stands behind the last token
    nt = torch.tensor([n], dtype=torch.int32, device=DEV)
    run_and_check(l, 6, "sigmoid", renorm=True, n=n, n_tokens=nt, want_scores=True)


def test_route_without_dispatch_and_with_given_outputs():
    l = logits_of(300, 64, torch.float32, 6)
    full = run_and_check(l, 4, "softmax")
    bare = moe.moe_topk_route(l, 4, dispatch=False)
    assert set(bare) == {"idx", "weights"}
    assert torch.equal(bare["idx"], full["idx"]) and torch.equal(bare["weights"], full["weights"])
    out = {n: torch.full_like(t, 77) for n, t in full.items()}
    ws = torch.full((moe.moe_topk_workspace_size(300, 64, 4),), 255, dtype=torch.uint8, device=DEV)
    got = moe.moe_topk_route(l, 4, out=out, workspace=ws)
    for name in out:
        assert got[name] is out[name] and torch.equal(got[name], full[name])
    assert moe.moe_device_status(ws) == (0, 0)
    with pytest.raises(ValueError):
        moe.moe_topk_route(l, 4, out={"scores": torch.empty(300, 64, device=DEV)})
    with pytest.raises(ValueError):
        moe.moe_topk_route(l, 4, out={"idx": torch.empty(300, 5, dtype=torch.int32, device=DEV)})
    with pytest.raises(ValueError):
        moe.moe_topk_route(l.t(), 4)
    with pytest.raises(moe.MoeError):
        moe.moe_topk_route(l, 4, workspace=ws[:256])
    with pytest.raises(moe.MoeError):
        moe.moe_topk_route(l, 65)


@pytest.mark.parametrize("T,dispatch", [(1, True), (40, True), (256, True), (300, True), (300, False), (6000, False)])
def test_route_writes_the_status_word_of_a_given_workspace(T, dispatch):
    l = logits_of(T, 64, torch.float32, 6)
    ws = torch.full((moe.moe_topk_workspace_size(T, 64, 4) or 256,), 0x40, dtype=torch.uint8, device=DEV)
    assert moe.moe_device_status(ws) == (6, 0x40404040)
    moe.moe_topk_route(l, 4, workspace=ws, dispatch=dispatch)
    assert moe.moe_device_status(ws) == (0, 0)
    if T <= 256 or not dispatch:                    # nothing else of it is used
        assert bool((ws[4:] == 0x40).all())
        for start, end in ((1, 200), (0, 3), (0, 0)):   # no status word fits there: left alone
            ws.fill_(0x40)
            moe.moe_topk_route(l, 4, workspace=ws[start:end], dispatch=dispatch)
            assert bool((ws == 0x40).all())


def test_route_empty_batch():
    l = torch.empty((0, 16), device=DEV)
    r = moe.moe_topk_route(l, 2)
    assert r["counts"].tolist() == [0] * 16 and r["offsets"].tolist() == [0] * 17 and r["idx"].shape == (0, 2)
    g = moe.moe_topk_route_backward(l, r["idx"], r["weights"])
    assert g.shape == (0, 16)


def test_route_matches_the_sublayers_router():
    # The same logits give the same choice and gates as moe_route_dispatch (E = 8, k = 2).
    from mixture_experts_ffn_14_b200 import expert_parallel as EP

    T, d = 150, 256
    x = torch.randn((T, d), generator=gen(11), device=DEV)
    wr = torch.zeros((d, 8), device=DEV)
    wr[torch.arange(8), torch.arange(8)] = 1.0      # logits = x[:, :8] exactly
    comp = EP.LibraryCompute(wr, torch.empty((8, d, 64), device=DEV), None, None)
    a = comp.route_dispatch(x)
    b = moe.moe_topk_route(x[:, :8].contiguous(), 2)
    for n, m in (("idx", "idx"), ("counts_dev", "counts"), ("offsets", "offsets"), ("perm_token", "perm_token"),
                 ("perm_slot", "perm_slot"), ("slot_pos", "slot_pos")):
        assert torch.equal(a[n], b[m]), n
    assert (a["gates"] - b["weights"]).abs().max() <= 120 * U   # both within 60 u of the exact value <= 1


# ------------------------------------------------------------------ backward --

def grad_bound(l, idx, gw, kind, renorm, scale, gs, n):
    """Bound of the fp32 error of each gradient: the roundings of one weight (weight_bound)
    on every term, and of the sums over the k chosen (k) and the E scores (37)."""
    T, E = l.shape
    lc, masked, s = ref.scores(l, kind)
    c = (120 + 2 * spread(l, idx) + idx.shape[1]
         + (np.minimum(np.where(masked, 0, np.abs(lc)).max(1, keepdims=True), 110) * 2 if kind == "softmax" else 0)) * U
    has = (idx >= 0) & (idx < E)
    g = np.where(has, np.abs(gw), 0) * abs(scale)
    size = np.zeros((T, E))
    p, _ = ref.weights_of(l, idx, kind, renorm, 1.0)
    each = p * (g + (g * p).sum(1, keepdims=True)) if renorm else g
    with np.errstate(over="ignore"):
        rest = 1 / (1 + np.exp(lc))
    ds = np.zeros((T, E)) if gs is None else np.abs(gs)
    direct = np.zeros((T, E))
    for t in range(T):
        for j in np.nonzero(has[t])[0]:
            (direct if renorm else ds)[t, idx[t, j]] += each[t, j]
    if kind == "sigmoid":
        size = s * rest * ds + direct * rest
    else:
        size = s * (ds + (s * ds).sum(1, keepdims=True)) + direct
    return c * size + 1e-36


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (33, 33, 5), (64, 60, 6), (100, 256, 8), (20, 512, 10), (17, 1000, 32)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(T, E, k, kind, renorm, dtype):
    l = logits_of(T, E, dtype, T + E + k, masked=0.2 if E > 8 else 0.0)
    l64 = l.double().cpu().numpy()
    g = gen(T * 7 + E)
    gw = torch.randn((T, k), generator=g, device=DEV)
    for gs in (None, torch.randn((T, E), generator=g, device=DEV)):
        n = T - T // 4
        idx = moe.moe_topk_route(l, k, score=SCORE[kind], dispatch=False)["idx"]
        got = moe.moe_topk_route_backward(l, idx, gw, score=SCORE[kind], renormalize=renorm, scale=1.5, grad_scores=gs,
                                          n_tokens=torch.tensor([n], dtype=torch.int32, device=DEV))
        a = (l64, idx.cpu().numpy(), gw.double().cpu().numpy(), kind, renorm, 1.5,
             None if gs is None else gs.double().cpu().numpy(), n)
        want = ref.route_backward(*a)
        lim = grad_bound(*a) + torch.finfo(dtype).eps / 2 * np.abs(want) * (0 if dtype == torch.float32 else 1.01)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= lim).all(), (err / lim).max()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(kind, renorm):
    T, E, k, h = 6, 12, 3, 1e-6
    l = logits_of(T, E, torch.float32, 77)
    l64 = l.double().cpu().numpy()
    idx = moe.moe_topk_route(l, k, score=SCORE[kind], dispatch=False)["idx"]
    gw, gs = (torch.randn(s, generator=gen(5), device=DEV) for s in ((T, k), (T, E)))
    got = moe.moe_topk_route_backward(l, idx, gw, score=SCORE[kind], renormalize=renorm, scale=2.0, grad_scores=gs)
    i, w, s = idx.cpu().numpy(), gw.double().cpu().numpy(), gs.double().cpu().numpy()

    def loss(x):
        a, b = ref.weights_of(x, i, kind, renorm, 2.0)
        return (a * w).sum(1) + (b * s).sum(1)

    num = np.zeros((T, E))
    for e in range(E):
        d = np.zeros((1, E))
        d[0, e] = h
        num[:, e] = (loss(l64 + d) - loss(l64 - d)) / (2 * h)
    # central differences: third derivatives below 10 times h^2, and 64-bit rounding of the loss over h
    lim = 10 * h * h + 20 * 2.0 ** -52 / h + grad_bound(l64, i, w, kind, renorm, 2.0, s, T)
    assert (np.abs(got.double().cpu().numpy() - num) <= lim).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(40, 33, 4), (40, 256, 8), (6000, 16, 3)])
def test_route_backward_reads_nothing_of_masked_and_padded_places(T, E, k, kind, renorm):
    l = logits_of(T, E, torch.float32, T + E, masked=0.4)
    n = T - T // 3
    nt = torch.tensor([n], dtype=torch.int32, device=DEV)
    idx = moe.moe_topk_route(l, k, score=SCORE[kind], dispatch=False, n_tokens=nt)["idx"]
    g = gen(T)
    gw, gs = torch.randn((T, k), generator=g, device=DEV), torch.randn((T, E), generator=g, device=DEV)
    want = moe.moe_topk_route_backward(l, idx, gw, score=SCORE[kind], renormalize=renorm, grad_scores=gs, n_tokens=nt)
    masked = ~(l > -float("inf"))
    assert bool((idx[:n] < 0).any()) and bool(masked[:n].any()) and not bool(torch.isnan(want).any())
    for odd in (float("nan"), float("inf")):
        gw[idx < 0], gs[masked] = odd, odd
        gs[n:] = odd
        gw[n:] = odd
        got = moe.moe_topk_route_backward(l, idx, gw, score=SCORE[kind], renormalize=renorm, grad_scores=gs, n_tokens=nt)
        assert torch.equal(got, want) and bool((got[masked] == 0).all()) and bool((got[n:] == 0).all())


def test_route_backward_odd_indices():
    # the same expert twice, and entries that are no expert
    l = logits_of(4, 16, torch.float32, 9)
    idx = torch.tensor([[3, 3, 5], [-1, 2, 16], [-5, -1, 1 << 30], [0, 15, 0]], dtype=torch.int32, device=DEV)
    gw = torch.randn((4, 3), generator=gen(2), device=DEV)
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            got = moe.moe_topk_route_backward(l, idx, gw, score=SCORE[kind], renormalize=renorm)
            a = (l.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64), gw.double().cpu().numpy(), kind, renorm, 1.0)
            want = ref.route_backward(*a)
            assert (np.abs(got.double().cpu().numpy() - want) <= grad_bound(*a, None, 4)).all(), (kind, renorm)


# ------------------------------------------------------------------- combine --

@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16], ids=["yf32", "ybf16"])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16], ids=["of32", "obf16"])
@pytest.mark.parametrize("T,k,d", [(1, 1, 8), (3, 2, 1032), (17, 3, 6144), (40, 8, 64), (5, 32, 256)])
@pytest.mark.parametrize("extras", [False, True])
def test_combine(T, k, d, yt, ot, extras):
    g = gen(T + k + d)
    R = T * k + 3
    y = torch.randn((R, d), generator=g, device=DEV).to(yt)
    pos = torch.randint(0, R, (T, k), generator=g, device=DEV, dtype=torch.int32)
    if extras:
        pos[torch.rand((T, k), generator=g, device=DEV) < 0.2] = -1
        pos[0, 0] = R                               # behind the last row
        pos[T - 1] = -7                             # a token with nothing
    y[R - 1] = float("nan")
    pos[pos == R - 1] = 0                           # a row that no slot names stays unread
    w = torch.rand((T, k), generator=g, device=DEV) if extras else None
    res = torch.randn((T, d), generator=g, device=DEV).to(ot) if extras else None
    got = moe.moe_combine_topk(y, pos, weights=w, residual=res, out_dtype=ot)
    num = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want, size = ref.combine(num(y), pos.cpu().numpy(), num(w), num(res))
    # k products and k additions, one rounding each; then the output's own
    lim = 2 * (k + 1) * U * size + torch.finfo(ot).eps / 2 * np.abs(want) * (0 if ot == torch.float32 else 1.01)
    assert (np.abs(num(got) - want) <= lim + 1e-37).all()
    if res is not None:                              # in place on the residual
        again = moe.moe_combine_topk(y, pos, weights=w, residual=res, out=res)
        assert again is res and torch.equal(res, got)


def test_combine_agrees_with_moe_combine_bitwise():
    from mixture_experts_ffn_14_b200 import expert_parallel as EP

    T, d = 25, 96
    y = torch.randn((2 * T, d), generator=gen(1), device=DEV)
    pos = torch.randperm(2 * T, generator=gen(2), device=DEV).to(torch.int32).reshape(T, 2).contiguous()
    comp = EP.LibraryCompute(None, torch.empty((1, 1, 1), device=DEV), None, None)
    want = comp.combine({"T": T, "dtype": moe.MOE_BF16, "slot_pos": pos}, y)
    assert torch.equal(moe.moe_combine_topk(y, pos, out_dtype=torch.bfloat16), want)


def test_combine_no_rows():
    out = moe.moe_combine_topk(torch.empty((0, 16), device=DEV), torch.zeros((3, 2), dtype=torch.int32, device=DEV))
    assert torch.equal(out, torch.zeros((3, 16), device=DEV))


# ------------------------------------------------------------ streams, graphs --

def test_route_on_other_streams_and_in_graphs():
    ls = [logits_of(T, 256, torch.bfloat16, T) for T in (300, 20)]
    bias = torch.randn(256, generator=gen(1), device=DEV) * 0.05
    kw = dict(score=moe.MOE_SCORE_SIGMOID, bias=bias, n_groups=8, topk_groups=4, group_rule=moe.MOE_GROUP_TOP2_SUM,
              renormalize=True)
    want = [moe.moe_topk_route(l, 8, **kw) for l in ls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[moe.moe_topk_route(l, 8, stream=s, **kw) for l, s in zip(ls, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(a[n], b[n]) for n in b)
    nt = torch.tensor([300], dtype=torch.int32, device=DEV)
    static = ls[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = moe.moe_topk_route(static, 8, n_tokens=nt, **kw)
        back = moe.moe_topk_route_backward(static, r["idx"], r["weights"], score=moe.MOE_SCORE_SIGMOID, renormalize=True,
                                           n_tokens=nt)
    for n, seed in ((300, 1), (7, 2), (0, 3), (299, 4)):
        static.copy_(logits_of(300, 256, torch.bfloat16, seed))
        nt.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        check(r, static, 8, "sigmoid", bias, 8, 4, "top2", True, 1.0, n)
        assert (back[n:] == 0).all() and bool(torch.isfinite(back).all())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,keep", [(64, 5, 1, 1), (256, 8, 1, 1), (256, 8, 8, 4), (40, 31, 1, 1), (33, 32, 1, 1),
                                             (96, 7, 3, 2), (512, 6, 16, 5)])
def test_route_single_near_ties(kind, E, k, groups, keep):
    """Values 0.01 apart but for one pair (or three, or a pair of groups) that fp32 cannot order."""
    g = gen(E + k)
    row = torch.randn(E, generator=g, device=DEV)
    _, _, s = ref.scores(row.double().cpu().numpy()[None], kind)
    order = torch.randperm(E, generator=g, device=DEV).cpu().numpy()
    for at in range(0, k + 3):
        for width in (2, 3):
            c = np.empty(E)
            c[order] = 5.0 - 0.01 * np.arange(E)
            if at + width <= E:
                c[order[at:at + width]] = c[order[at]]
            if groups > 1 and at % 2:
                # two groups of the same largest pair of values
                gs = E // groups
                a, b = (order[at] // gs) * gs, (order[(at + 9) % E] // gs) * gs
                c[b:b + 2] = np.sort(c[a:a + gs])[::-1][:2]
            bias = torch.from_numpy((c - s[0]).astype(np.float32)).to(DEV)
            for rule in ("max", "top2") if groups > 1 else ("max",):
                run_and_check(row[None].contiguous(), k, kind, bias=bias, groups=groups, keep=keep, rule=rule)
            # the same for logits alone, one step of fp32 apart
            l = torch.from_numpy(np.round(c * 2 ** 20).astype(np.float32) / 2 ** 20).to(DEV)
            if at + width <= E:
                e = torch.tensor(order[at:at + width], device=DEV)
                l[e] += torch.arange(width, device=DEV) * 2.0 ** -21
            run_and_check(l[None].contiguous(), k, kind, groups=groups, keep=keep, rule="max")


def test_binding_refuses_what_the_c_types_would_cut():
    logits = torch.zeros((4, 8), device=DEV)
    for bad in (dict(k=2 ** 32 + 2), dict(k=2, n_groups=2 ** 40), dict(k=2, out=[]), dict(k=2, bias=[0.0] * 8),
                dict(k=2, out={"idx": torch.zeros((4, 2), dtype=torch.int32, device=DEV), "other": None})):
        with pytest.raises(ValueError):
            moe.moe_topk_route(logits, **bad)
    with pytest.raises(TypeError):
        moe.moe_topk_route(logits, 2.5)
    with pytest.raises(ValueError):
        moe.moe_topk_route(logits, 2, workspace=torch.zeros(256, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_topk_route(logits, 9)
    kept = torch.full((4, 2), 5, dtype=torch.int32, device=DEV)
    r = moe.moe_topk_route(logits, 2, out={"idx": kept, "weights": None}, dispatch=False)
    assert r["idx"] is kept and list(r) == ["idx", "weights"]
    assert kept.tolist() == [[0, 1]] * 4


def test_binding_allocates_on_the_stream_it_is_given():
    y, pos = torch.ones((64, 64), device=DEV), torch.arange(64, dtype=torch.int32, device=DEV).view(32, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        out = moe.moe_combine_topk(y, pos, stream=stream)
        side.synchronize()
        assert bool((out == 2).all()) and torch.cuda.current_stream() != side


# Group sizes that are no powers of two, groups with idle lanes, more than 8 registers per
# lane, and the two that do not fit runs of lanes (9 x 113, 24 x 40).
ODD_GROUPS = [(136, 8, 3), (88, 8, 6), (44, 4, 2), (100, 5, 2), (6, 2, 1), (250, 2, 1), (348, 4, 3), (504, 8, 6),
              (512, 8, 6), (960, 24, 7), (1017, 9, 4), (31, 31, 5), (693, 11, 5)]


@pytest.mark.parametrize("E,groups,keep", ODD_GROUPS)
@pytest.mark.parametrize("rule", ["max", "top2"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_route_groups_of_odd_sizes(E, groups, keep, rule, kind, dtype):
    k = min(9, E // groups * keep)
    for masked, T in ((0.2, 200), (0.9, 33)):
        l = logits_of(T, E, dtype, E + groups, masked=masked)
        for bias in (None, torch.randn(E, generator=gen(E), device=DEV) * 0.1):
            run_and_check(l, k, kind, bias=bias, groups=groups, keep=keep, rule=rule, renorm=dtype == torch.bfloat16,
                          want_scores=T == 33)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep", [(136, 8, 3), (512, 8, 6), (504, 8, 3), (1024, 4, 2), (100, 5, 2), (960, 24, 7)])
def test_route_near_ties_in_groups_of_odd_sizes(kind, E, groups, keep):
    """score + bias equal up to the rounding of the bias, in every expert, in a few, and in the two
    largest of each group."""
    k, gs = 6, E // groups
    g = gen(E)
    row = torch.randn(E, generator=g, device=DEV)
    _, _, s = ref.scores(row.double().cpu().numpy()[None], kind)
    order = torch.randperm(E, generator=g, device=DEV).cpu().numpy()
    flat = np.ones(E)
    few = 3.0 - 0.01 * order
    few[order[:5]] = few[order[0]]
    heads = 1.0 - 0.01 * (np.arange(E) % gs)
    heads[np.arange(E) % gs == min(1, gs - 1)] = 1.0
    for c in (flat, few, heads):
        bias = torch.from_numpy((c - s[0]).astype(np.float32)).to(DEV)
        for rule in ("max", "top2"):
            run_and_check(row.repeat(3, 1), k, kind, bias=bias, groups=groups, keep=keep, rule=rule)
    l = torch.from_numpy(few.astype(np.float32)).to(DEV).repeat(2, 1)
    l[1] += torch.arange(E, device=DEV) * 2.0 ** -21
    for rule in ("max", "top2"):
        run_and_check(l, k, kind, groups=groups, keep=keep, rule=rule)
