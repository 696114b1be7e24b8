"""moe_int8_product on the GPU against the definition in 64 bits. The integer sums are
exact in both, so the bounds count the fp32 roundings behind them (u = 2^-24) and the
rounding of the output's type."""

import math

import pytest
import torch

import _routed_reference as ref
import mixture_experts_ffn_14_b200 as moe
from _int8_plan import CASES, form

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
ACT = {"gelu": moe.MOE_ACT_GELU_TANH, "erf": moe.MOE_ACT_GELU_ERF, "silu": moe.MOE_ACT_SILU}


def make(R, K, N, n, seed, x="bf16", pair=False, rows=None, gate=False, tokens=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = {"K": K, "N": N, "n": n, "R": R}
    if x == "i8":
        c["x"] = torch.randint(-128, 128, (R, K), generator=g, device=DEV, dtype=torch.int8)
        c["x_scale"] = torch.rand(R, generator=g, device=DEV) * 0.02
    else:
        c["x"] = torch.randn((tokens or R, K), generator=g, device=DEV).to(
            torch.bfloat16 if x == "bf16" else torch.float32)
        c["x_scale"] = None
    c["index"] = torch.randint(0, tokens, (R,), generator=g, device=DEV, dtype=torch.int32) if tokens else None
    c["counts"] = None if rows is None else torch.tensor(rows, dtype=torch.int32, device=DEV)
    c["rows"] = [R] if rows is None else list(rows)
    w = lambda: torch.randint(-128, 128, (n, K, N), generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    s = lambda: ((torch.rand((n, N), generator=g, device=DEV) + 0.5) / (90 * math.sqrt(K))).to(torch.bfloat16)  # noqa: E731
    c["w"], c["s"] = w(), s()
    c["w_up"], c["s_up"] = (w(), s()) if pair else (None, None)
    c["gate"] = torch.rand(R, generator=g, device=DEV) if gate else None
    return c


def call(c, **kw):
    return moe.moe_int8_product(c["x"], c["w"], c["s"], x_scale=c["x_scale"], index=c["index"], counts=c["counts"],
                                w_up=c["w_up"], s_up=c["s_up"], gate=c["gate"], **kw)


def quantised(c):
    """(q, a) of the rows in 64 bits: a is the fp32 quotient of the definition."""
    x = c["x"]
    if c["x_scale"] is not None:
        return x.double(), c["x_scale"].double()
    if c["index"] is not None:
        i = c["index"].long()
        real = (i >= 0) & (i < x.shape[0])
        x = torch.where(real[:, None], x[torch.where(real, i, 0)], torch.zeros((), dtype=x.dtype, device=DEV))
    x = x.double()
    top = x.abs().amax(1)
    top = torch.where(torch.isfinite(x).all(1), top, math.nan)
    q = torch.round(127 * x / torch.where(top > 0, top, 1.0)[:, None])
    q[~(top > 0)] = 0
    return q, (top / 127).float().double()  # divided in 64 bits: the fp32 quotient, rounded once


def act64(z, act):
    if act == "silu":
        return z * torch.special.expit(z), z, torch.ones_like(z)
    if act == "erf":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5)), z * z, 2 * z
    t = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.special.expit(t), t, 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def reference(c, act="gelu"):
    """(rows 0 .. sum of counts of the result, bound of the fp32 error)."""
    q, a = quantised(c)
    outs, lims, at = [], [], 0
    for e, m in enumerate(c["rows"]):
        r = slice(at, at + m)
        at += m
        z = (q[r] @ c["w"][e].double()) * a[r, None] * c["s"][e].double()
        # integer -> fp32, row scale, channel scale: one rounding each (and the gate's)
        lim = 4 * U * z.abs()
        if c["w_up"] is not None:
            y, t, dt = act64(z, act)
            z1 = (q[r] @ c["w_up"][e].double()) * a[r, None] * c["s_up"][e].double()
            # act: three roundings of z through |z t'|, the argument (4 u |t|, in the exponent), the exponential
            # (2 + 1.2 |t| ulp) or erfc (4 ulp, its argument's roundings through 2 t), sum, quotient 2 ulp
            rel = 2 * U * (12 + 4 * (1 + (z * dt).abs()) + 8 * t.abs())
            z, lim = y * z1, (y * z1).abs() * (rel + 8 * U) + 1e-30
        if c["gate"] is not None:
            z, lim = z * c["gate"][r, None].double(), lim * c["gate"][r, None].double()
        outs.append(z)
        lims.append(lim)
    return torch.cat(outs), torch.cat(lims)


def check(c, got, act="gelu", tail=None):
    want, lim = reference(c, act)
    m = want.shape[0]
    g = got[:m].double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan)
    half = 0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    err = torch.where(nan, 0.0, (g - want).abs())
    lim = torch.where(nan, 1.0, lim * 1.01 + half * (want.abs() + lim)) + 1e-36
    assert bool((err <= lim).all()), (float((err / lim).max()), torch.nonzero(err > lim)[:5].tolist())
    if tail is not None:
        assert bool((got[m:] == tail).all())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["obf16", "of32"])
@pytest.mark.parametrize("x", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("R,K,N,rows", [
    (1, 16, 16, None), (1, 2048, 512, None), (3, 144, 272, [2, 1]), (17, 128, 128, [0, 17, 0]), (64, 256, 512, [8] * 8),
    (65, 6144, 144, [1, 63, 1]), (129, 1040, 2064, None), (333, 512, 400, None), (200, 4096, 1040, [100, 0, 30, 70, 0]),
    (700, 640, 272, [10, 450, 0, 240]), (700, 640, 4112, [10, 450, 0, 240]), (1300, 640, 2064, None),
    (1811, 272, 1552, [700, 0, 1111]), (1600, 1040, 2064, [1, 512, 1087])])
@pytest.mark.parametrize("pair", [False, True])
def test_sizes(R, K, N, rows, x, out, pair):
    c = make(R, K, N, len(rows) if rows else 1, R + K + N, x=x, pair=pair, rows=rows, gate=R % 2 == 1)
    check(c, call(c, out_dtype=out))


@pytest.mark.parametrize("K", [2176, 6144])     # whole tiles, and tiles cut into runs of K blocks
@pytest.mark.parametrize("R,N,rows", [(20, 8192, [5, 0, 15]), (20, 19216, [5, 0, 15]), (290, 4624, [100, 128, 2, 60])])
@pytest.mark.parametrize("pair", [False, True])
def test_tiles_of_several_ctas(R, N, rows, K, pair):
    c = make(R, K, N, len(rows), R + N, pair=pair, rows=rows, tokens=11)
    ws = torch.empty(moe.moe_int8_workspace_size(R, K, N, len(rows), moe.MOE_BF16, pair), dtype=torch.uint8, device=DEV)
    outs = [call(c, workspace=ws) for _ in range(3)]      # one workspace, one call after the other
    check(c, outs[0])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("x,out", [("bf16", torch.bfloat16), ("f32", torch.float32), ("i8", torch.float32)])
@pytest.mark.parametrize("name,tile,R,K,N,rows,pair", CASES,
                         ids=[f"{c[0]}{c[1]}-{c[2]}x{c[3]}x{c[4]}-{'gated' if c[6] else 'plain'}" for c in CASES])
def test_every_form(name, tile, R, K, N, rows, pair, x, out):
    assert form(R, K, N, len(rows), x, pair)[:2] == (name, tile)
    c = make(R, K, N, len(rows), R + K + N + len(rows), x=x, pair=pair, rows=rows, gate=True)
    o = torch.full((R, N), 7.0, device=DEV, dtype=out)
    first = call(c, out=o).clone()
    check(c, o, tail=7.0)
    # the sums are integers: whatever order the tiles and their parts come in, the same bits
    for _ in range(3):
        assert torch.equal(call(c, out=o.fill_(7.0)), first)


@pytest.mark.parametrize("act", ["gelu", "erf", "silu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["obf16", "of32"])
def test_activations(act, out):
    c = make(90, 512, 256, 2, 5, pair=True, rows=[40, 50], gate=True)
    c["s"] = (c["s"].float() * 4).to(torch.bfloat16)     # gate values out to +-15
    check(c, call(c, out_dtype=out, activation=ACT[act]), act)


@pytest.mark.parametrize("act", ["gelu", "erf", "silu"])
@pytest.mark.parametrize("R,n", [(40, 2), (700, 2)])
def test_gate_values_whose_square_leaves_the_fp32_range(R, n, act):
    c = make(R, 256, 272, n, 31, x="f32", pair=True, rows=[R // 2, R - R // 2])
    c["x"] *= 1e25
    c["s_up"] = (c["s_up"].float() * 1e-30).to(torch.bfloat16)
    got = call(c, out_dtype=torch.float32, activation=ACT[act]).double()
    q, a = quantised(c)
    for e, r in enumerate((slice(0, R // 2), slice(R // 2, R))):
        z = (q[r] @ c["w"][e].double()) * a[r, None] * c["s"][e].double()
        z1 = (q[r] @ c["w_up"][e].double()) * a[r, None] * c["s_up"][e].double()
        assert float(z.abs().max()) > 2.0 ** 64
        # far from 0 every activation is z or 0 to the last bit; left are the roundings of an integer to fp32
        # and of two scales, twice, of the activation's own steps (reciprocal 2 u, product u) and of the product
        want = torch.where(z > 0, z, 0.0) * z1
        sure = z.abs() > 1e3
        assert int(sure.sum()) > 0.9 * sure.numel()
        err = (got[r] - want).abs()
        assert bool((err[sure] <= 12 * U * want.abs()[sure]).all()) and not bool(torch.isnan(got[r]).any())


@pytest.mark.parametrize("act", ["gelu", "erf", "silu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["obf16", "of32"])
@pytest.mark.parametrize("R,N", [(40, 16), (40, 4112), (110, 20000), (700, 272), (1400, 4112)])
def test_gate_values_of_infinity(R, N, out, act):
    # act(+inf) = +inf, act(-inf) = -inf * 0, a NaN, times an up value of 127 * 64 * 1e-36 * 1e38 (8e5)
    K = 64
    x = torch.full((R, K), 1e38, device=DEV)
    x[1::2] *= -1
    w = torch.full((1, K, N), 127, dtype=torch.int8, device=DEV)
    w[:, :, 3::4] = -127
    s = torch.full((1, N), 1e4, device=DEV, dtype=torch.bfloat16)
    su = torch.full((1, N), 1e-36, device=DEV, dtype=torch.bfloat16)
    got = moe.moe_int8_product(x, w, s, w_up=w.abs(), s_up=su, activation=ACT[act], out_dtype=out)
    z = x[:, :1] * w[0, :1]                          # its sign is the gate value's; the up value has the row's
    assert torch.equal(torch.isnan(got), z < 0)
    want = torch.where(x[:, :1] > 0, math.inf, -math.inf).expand(R, N)
    assert torch.equal(got[z > 0].float(), want[z > 0])


@pytest.mark.parametrize("R,rows", [(40, [5, 0, 7, 20]), (600, [200, 0, 100, 150])])
def test_rows_behind_the_last_expert_stay(R, rows):
    c = make(R, 272, 144, 4, R, rows=rows, tokens=33)
    out = torch.full((R, 144), 7.0, device=DEV)
    check(c, call(c, out=out), tail=7.0)
    # an output that is not given starts as zeros there
    check(c, call(c, out_dtype=torch.float32), tail=0.0)


def test_gathered_rows():
    c = make(300, 640, 512, 3, 11, rows=[100, 150, 50], tokens=40, pair=True)
    c["index"][::7] = -1
    c["index"][3] = 40
    c["index"][4] = 1 << 30
    check(c, call(c, out_dtype=torch.float32))
    c["index"] = torch.zeros_like(c["index"])      # the same row every time
    check(c, call(c, out_dtype=torch.float32))


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("K", [48, 2048, 5120, 33024])   # one, a few, many values per thread, and rows read twice
def test_odd_rows(x, K):
    c = make(12, K, 32, 1, K, x=x)
    v = c["x"]
    v[0] = 0
    v[1, K // 2] = math.nan
    v[2, 0] = math.inf
    v[3, K - 1] = -math.inf
    v[4] *= 1e-38                                   # scales below the fp32 normal range
    v[5] *= 1e37
    v[6] = 0
    v[6, 5] = torch.finfo(v.dtype).smallest_normal
    v[7] = (torch.arange(K, device=DEV) % 255 - 127).to(v.dtype)         # integers: quotients on halves
    v[7, 0] = 254
    v[8] = 1
    v[9, 3] = torch.finfo(v.dtype).max
    v[10] = v[10] * 0 - 0.0
    c["s"] = torch.ones_like(c["s"])
    got = call(c, out_dtype=torch.float32)
    want, lim = reference(c)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and bool(nan[1:4].all()) and int(nan.any(1).sum()) == 3
    # what lies past the largest fp32 (rows 5 and 9) becomes an infinity of its sign
    over = want.abs() >= 2.0 ** 128
    assert torch.equal(got[over], torch.sign(want[over]).float() * math.inf)
    # below the normal range a rounding is half of 2^-149, of the scale and then of each product
    err, lim = (got.double() - want).abs(), lim + 2.0 ** -148 * (K * 127 * 128 + 2)
    # a value whose bound reaches the border of overflow, half a step above the largest fp32, may be
    # either (127 * (max / 127) is one)
    border = (want.abs() + lim >= (2 - 2.0 ** -24) * 2.0 ** 127) & (got == torch.sign(want).float() * math.inf)
    bad = ~((err <= lim) | nan | over | border)
    assert not bool(bad.any()), torch.nonzero(bad)[:5].tolist()
    assert bool((got[0] == 0).all()) and bool((got[10] == 0).all())


def test_largest_sums():
    # K = 131056: every product 128 * 128, the sum 2147221504 just inside 32 bits
    K = 131056
    c = make(5, K, 32, 1, 1, x="i8")
    c["x"].fill_(-128)
    c["w"].fill_(-128)
    c["w"][:, :, 1::2] = 127
    c["x_scale"].fill_(1.0)
    c["s"].fill_(1.0)
    got = call(c, out_dtype=torch.float32)
    want = torch.tensor([K * 128 * 128, -K * 128 * 127] * 16, dtype=torch.float64, device=DEV).float()
    assert torch.equal(got, want.expand(5, 32))


@pytest.mark.parametrize("x", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 2048, 33024])   # rows that pass through shared memory, and rows read twice
def test_rows_of_an_index_that_names_none(x, K):
    # x without a single row: there is no address that may be read
    R, N = 6, 48
    w = torch.randint(-128, 128, (1, K, N), device=DEV, dtype=torch.int8)
    s = torch.ones((1, N), device=DEV, dtype=torch.bfloat16)
    index = torch.tensor([-1, 0, 7, -(2 ** 31), 2 ** 31 - 1, 1], dtype=torch.int32, device=DEV)
    out = torch.full((R, N), 3.0, device=DEV)
    moe.moe_int8_product(torch.empty((0, K), dtype=x, device=DEV), w, s, index=index, out=out)
    assert bool((out == 0).all())
    # and beside rows that are there
    c = make(R, K, N, 1, K, x="bf16" if x == torch.bfloat16 else "f32", tokens=2)
    c["index"] = index
    check(c, call(c, out_dtype=torch.float32))


def test_many_experts():
    n = 1000
    rows = [(e * 7) % 5 for e in range(n)]
    c = make(sum(rows) + 9, 64, 48, n, 3, rows=rows, pair=True)
    out = torch.full((c["R"], 48), 3.0, device=DEV, dtype=torch.bfloat16)
    check(c, call(c, out=out), tail=3.0)


def test_no_rows_at_all():
    c = make(20, 64, 48, 3, 3, rows=[0, 0, 0])
    out = torch.full((20, 48), 3.0, device=DEV)
    assert bool((call(c, out=out) == 3.0).all())
    e = moe.moe_int8_product(torch.empty((0, 64), device=DEV), c["w"], c["s"], counts=c["counts"])
    assert e.shape == (0, 48)


@pytest.mark.parametrize("counts", [[30, 30], [-5, 20], [2**31 - 1, 2**31 - 1], [0, 41]])
def test_bad_counts_are_cut_and_reported(counts):
    c = make(40, 64, 48, 2, 3, rows=counts)
    ws = torch.empty(moe.moe_int8_workspace_size(40, 64, 48, 2), dtype=torch.uint8, device=DEV)
    out = torch.full((60, 48), 3.0, device=DEV)
    moe.moe_int8_product(c["x"], c["w"], c["s"], counts=c["counts"], out=out[:40], workspace=ws)
    assert moe.moe_device_status(ws) == (6, 0x40)
    assert bool((out[40:] == 3.0).all())
    m0 = min(max(counts[0], 0), 40)
    m1 = min(max(counts[1], 0), 40 - m0)
    c["rows"] = [m0, m1]
    check(c, out[:40], tail=3.0)
    c = make(40, 64, 48, 2, 3, rows=[20, 20])
    moe.moe_int8_product(c["x"], c["w"], c["s"], counts=c["counts"], out=out[:40], workspace=ws)
    assert moe.moe_device_status(ws) == (0, 0)
    check(c, out[:40])


def test_binding_refuses():
    c = make(40, 64, 48, 2, 3, rows=[20, 20])
    for bad in (dict(counts=c["counts"].long()), dict(gate=torch.ones(39, device=DEV)),
                dict(out=torch.empty((39, 48), device=DEV)), dict(out=torch.empty((40, 48), device=DEV).half()),
                dict(counts=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            moe.moe_int8_product(c["x"], c["w"], c["s"], **{"counts": c["counts"], **bad})
    with pytest.raises(ValueError):
        moe.moe_int8_product(c["x"].t().contiguous().t(), c["w"], c["s"], counts=c["counts"])
    with pytest.raises(moe.MoeError):
        moe.moe_int8_product(c["x"], c["w"], c["s"])
    with pytest.raises(moe.MoeError):
        moe.moe_int8_product(c["x"], c["w"], c["s"], counts=c["counts"],
                             workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_binding_refuses_other_shapes_of_index():
    c = make(40, 64, 48, 1, 3)
    for index in (torch.tensor(3, dtype=torch.int32, device=DEV), torch.zeros((2, 20), dtype=torch.int32, device=DEV)):
        with pytest.raises(ValueError):
            moe.moe_int8_product(c["x"], c["w"], c["s"], index=index)


def test_streams_and_graph():
    cs = [make(40, 512, 272, 2, 21, rows=[20, 20]), make(700, 640, 272, 2, 22, rows=[300, 400], pair=True)]
    want = [call(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[call(c, stream=s) for c, s in zip(cs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a, b)
    c = make(300, 256, 144, 3, 23, rows=[100, 100, 100])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(c)
    for seed, rows in ((1, [300, 0, 0]), (2, [1, 150, 149]), (3, [0, 0, 300])):
        d = make(300, 256, 144, 3, seed, rows=rows)
        for name in ("x", "w", "s", "counts"):
            c[name].copy_(d[name])
        c["rows"] = rows
        graph.replay()
        torch.cuda.synchronize()
        check(c, out)


@pytest.mark.parametrize("T,d,f,E,k,kind", [(1, 256, 384, 8, 2, "softmax"), (50, 256, 384, 8, 2, "softmax"),
                                            (300, 512, 256, 24, 6, "sigmoid"), (700, 256, 640, 16, 3, "sigmoid")])
def test_one_layer_of_the_operators_together(T, d, f, E, k, kind):
    """route -> gate/up -> down -> combine, each step against its own 64-bit value on the
    inputs it was given, and the layer against the layer in 64 bits."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    x = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device=DEV)
    i8 = lambda *s: torch.randint(-127, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    sc = lambda n, m, fan: ((torch.rand((n, m), generator=g, device=DEV) + 0.5) / (127 * math.sqrt(fan))).to(torch.bfloat16)  # noqa: E731
    wg, wu, wd = i8(E, d, f), i8(E, d, f), i8(E, f, d)
    sg, su, sd = sc(E, f, d), sc(E, f, d), sc(E, d, f)
    n = T - T // 5
    nt = torch.tensor([n], dtype=torch.int32, device=DEV)
    r = moe.moe_topk_route(logits, k, score=moe.MOE_SCORE_SIGMOID if kind == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                           renormalize=True, n_tokens=nt)
    h = moe.moe_int8_product(x, wg, sg, index=r["perm_token"], counts=r["counts"], w_up=wu, s_up=su)
    y = moe.moe_int8_product(h, wd, sd, counts=r["counts"], gate=r["gate_perm"], out_dtype=torch.float32)
    out = moe.moe_combine_topk(y, r["slot_pos"], out_dtype=torch.bfloat16)
    rows = r["counts"].tolist()
    assert sum(rows) == n * k
    check({"x": x, "x_scale": None, "index": r["perm_token"], "rows": rows, "w": wg, "s": sg, "w_up": wu, "s_up": su,
           "gate": None}, h)
    check({"x": h, "x_scale": None, "index": None, "rows": rows, "w": wd, "s": sd, "w_up": None, "s_up": None,
           "gate": r["gate_perm"]}, y)
    assert bool((out[n:] == 0).all())
    # the layer without rounding anything to 8 or 16 bits on the way
    want = torch.zeros((T, d), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(want)
    for t in range(0, n, max(1, n // 25)):
        for j in range(k):
            e = int(r["idx"][t, j])
            xt = x[t].double()
            z, z1 = xt @ (wg[e].double() * sg[e].double()), xt @ (wu[e].double() * su[e].double())
            hh = act64(z, "gelu")[0] * z1
            p = hh @ (wd[e].double() * sd[e].double()) * float(r["weights"][t, j])
            want[t] += p
            # a value's rounding to 8 bits is at most max/254 off; the errors of the sums' terms are
            # independent, so their root mean square counts, with a factor 8 for the largest of all
            size[t] += float(r["weights"][t, j]) * (xt.abs().max() / 254 * 2 + hh.abs().max() / 254)
        assert bool(((out[t].double() - want[t]).abs() <= 8 * size[t] + want[t].abs() * 2.0 ** -8).all())


def failing(c, got):
    """Share of the elements of the result that check() would refuse."""
    want, lim = reference(c)
    half = 0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    err = (got[:want.shape[0]].double() - want).abs()
    return float((err > lim * 1.01 + half * (want.abs() + lim) + 1e-36).double().mean())


@pytest.mark.parametrize("T,d,f,E,k,kind", [(1, 256, 384, 8, 2, "softmax"), (50, 256, 384, 8, 2, "softmax"),
                                            (300, 512, 256, 24, 6, "sigmoid"), (700, 256, 640, 16, 3, "sigmoid")])
def test_one_layer_against_a_choice_and_an_order_made_in_64_bits(T, d, f, E, k, kind):
    """The same layer, every step against its 64-bit value from what the step before it
    left, but at the experts, weights and places of a routing in 64 bits, not of the call's own
    arrays: a row at another place, of another token, expert or slot is refused."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T + 1)
    x = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device=DEV)
    i8 = lambda *s: torch.randint(-127, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    sc = lambda n, m, fan: ((torch.rand((n, m), generator=g, device=DEV) + 0.5) / (127 * math.sqrt(fan))).to(torch.bfloat16)  # noqa: E731
    wg, wu, wd = i8(E, d, f), i8(E, d, f), i8(E, f, d)
    sg, su, sd = sc(E, f, d), sc(E, f, d), sc(E, d, f)
    n = T - T // 5
    r = moe.moe_topk_route(logits, k, score=moe.MOE_SCORE_SIGMOID if kind == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                           renormalize=True, n_tokens=torch.tensor([n], dtype=torch.int32, device=DEV))
    h = moe.moe_int8_product(x, wg, sg, index=r["perm_token"], counts=r["counts"], w_up=wu, s_up=su)
    y = moe.moe_int8_product(h, wd, sd, counts=r["counts"], gate=r["gate_perm"], out_dtype=torch.float32)
    out = moe.moe_combine_topk(y, r["slot_pos"], out_dtype=torch.bfloat16)

    want = ref.route(logits.double().cpu().numpy(), k, kind, renorm=True, n=n)
    # the weights: 20 roundings and two for each unit that a row's logits span (below 12 here)
    w = r["weights"].double().cpu().numpy()
    assert (abs(w - want["weights"]) <= 44 * U * want["weights"]).all()
    rows, m = want["counts"].tolist(), n * k
    token, slot = (torch.from_numpy(want[name]).to(DEV) for name in ("perm_token", "perm_slot"))
    gate = torch.zeros(T * k, device=DEV)
    gate[:m] = r["weights"][token[:m], slot[:m]]
    up = {"x": x, "x_scale": None, "index": token.int(), "rows": rows, "w": wg, "s": sg, "w_up": wu, "s_up": su,
          "gate": None}
    down = {"x": h, "x_scale": None, "index": None, "rows": rows, "w": wd, "s": sd, "w_up": None, "s_up": None,
            "gate": gate}
    check(up, h, tail=0.0)
    check(down, y, tail=0.0)
    pos = torch.from_numpy(want["slot_pos"]).to(DEV)

    def combined(pos):
        part = torch.where((pos >= 0)[:, :, None], y.double()[pos.clamp(min=0)], 0.0)
        total = part.sum(1)
        # k additions, then the rounding to 16 bits
        return total, 2 * k * U * part.abs().sum(1) + 2.0 ** -8 * 1.01 * total.abs() + 1e-37

    total, lim = combined(pos)
    assert bool(((out.double() - total).abs() <= lim).all()) and bool((out[n:] == 0).all())
    # what these bounds refuse: nothing at all, and each kind of exchange
    assert float((total[:n].abs() > lim[:n]).double().mean()) > 0.99
    assert failing(up, torch.zeros_like(h)) > 0.9 and failing(down, torch.zeros_like(y)) > 0.9
    if n > 1:
        assert failing({**up, "index": token.int().roll(1)}, h) > 0.9
        other, lim = combined(torch.cat([pos[:n].roll(1, 0), pos[n:]]))
        assert float(((out.double() - other).abs() > lim)[:n].double().mean()) > 0.9
        swapped = torch.zeros_like(gate)
        swapped[:m] = r["weights"].roll(1, 1)[token[:m], slot[:m]]
        assert failing({**down, "gate": swapped}, y) > 0.9
        assert failing({**down, "w": wd.roll(1, 0)}, y) > 0.9
