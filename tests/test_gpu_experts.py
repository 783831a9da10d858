"""GPU tests of the expert-layer operators (route, quantize_rows, i8_matmul, experts) against
plain 64-bit forms (tests/experts_ref.py): sizes from one to odd and long, every type, rows
without an expert, ties, infinities and NaN, strides, other streams, graph replays.

Tolerances, each from the roundings made (u = 2^-24, half a step of fp32):
 - choices, whole numbers and scales of 8-bit rows are equal;
 - i8_matmul: sum -> fp32, scale product, product, bias: 4 u (|p| + |b|), then half a step of
   the output type (eps / 2 of the value, or of the smallest normal for subnormal values);
 - experts: per slot 3 u for the scaled sum and 1 u for the weight, k u for the sum of k slots:
   (k + 4) u sum |w p|, then half a step of the output type;
 - route weights: evaluated in fp32 at worst: the exponent's argument x = l - max is off by
   u |x| and its exponential by 2 u, the sum (10 levels of pairs and up to 16 terms a lane) by
   26 u plus the worst term, two divisions and the scale by 1 u each, the sum of the chosen by
   64 u more: (2 max|x| + 100) u relative."""
import math

import numpy as np
import pytest
import torch

import experts_ref as ref
from gpu_util import say, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def P():
    import activation_sparse_decode_rank_amd as P  # fails loudly without the HIP library
    torch.cuda.init()
    yield P


def rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(y, dtype):
    """Half a step of the type at y (its smallest normal below that)."""
    fi = torch.finfo(dtype)
    return fi.eps / 2 * np.maximum(np.abs(y), fi.tiny)


def check(got, want, err, dtype):
    got = f64(got)
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(got), bad)
    d = np.abs(got - want)[~bad]
    lim = (err + half_step(np.abs(want) + err, dtype))[~bad]
    assert (d <= lim).all(), f"{int((d > lim).sum())} values off, worst {np.max(d / lim):.3g} of the bound"


# ------------------------------------------------------------------------------------ route
def logits_of(T, E, dtype, seed, kind="normal"):
    g = rng(1, T, E, seed)
    l = g.standard_normal((T, E)) * 2
    if kind == "ties":
        l = g.integers(-2, 3, (T, E)).astype(np.float64)
    if kind == "masked":
        l[g.random((T, E)) < 0.6] = -np.inf
        l[g.random((T, E)) < 0.05] = np.nan
        l[g.random((T, E)) < 0.02] = np.inf
        l[::3] = -np.inf
        l[1::7] = np.nan
    if kind == "far":
        l *= 200
    return dev(l, DT[dtype])


def check_route(P, l, k, **kw):
    bias = kw.pop("bias", None)
    idx, w = P.route(l, k, bias=bias, **kw)
    kw["renorm"] = kw.pop("renormalize", True)
    ri, rw = ref.route(f64(l), k, bias=None if bias is None else to_np(bias), **kw)
    assert np.array_equal(to_np(idx), ri)
    x = np.where(np.isfinite(f64(l)), f64(l), 0.0)
    far = np.minimum(2 * np.abs(x).max(initial=0.0), 110.0)  # e^-104 is the smallest fp32 value
    lim = (2 * far + 100) * U * np.abs(rw) + 2.0 ** -126 * abs(kw.get("scale", 1.0))
    assert (np.abs(f64(w) - rw) <= lim).all(), float(np.max(np.abs(f64(w) - rw) / lim))
    return idx, w


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (3, 3), (8, 2), (63, 5), (64, 8), (65, 64), (128, 1),
                                 (160, 6), (256, 8), (384, 8), (513, 7), (1024, 64), (1000, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_sizes(P, E, k, score):
    say("route", E, k, score)
    for T, dt in ((1, "f32"), (5, "f16"), (131, "bf16")):
        check_route(P, logits_of(T, E, dt, k), k, score=score)
        b = dev(rng(2, E, k).standard_normal(E) * 0.1)
        check_route(P, logits_of(T, E, dt, k + 1), k, score=score, bias=b, renormalize=False, scale=2.5)


@pytest.mark.parametrize("E,groups,top_groups", [(8, 4, 2), (64, 8, 3), (256, 8, 4), (160, 5, 5), (320, 64, 7),
                                                 (1024, 2, 1), (63, 63, 9), (12, 3, 1)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
def test_route_groups(P, E, groups, top_groups, group_top, kind):
    say("route groups", E, groups, top_groups, group_top, kind)
    kw = dict(groups=groups, top_groups=top_groups, group_top=group_top)
    for score, bias in (("softmax", False), ("sigmoid", True), ("softmax", True), ("sigmoid", False)):
        b = dev(rng(3, E).integers(-1, 2, E) * 0.25) if bias else None
        check_route(P, logits_of(37, E, "f32", groups, kind), min(E, 6), score=score, bias=b, **kw)


@pytest.mark.parametrize("kind", ["ties", "masked", "far"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_route_ties_and_masks(P, kind, score, dtype):
    say("route", kind, score, dtype)
    for E, k in ((8, 4), (64, 64), (200, 12)):
        check_route(P, logits_of(70, E, dtype, k, kind), k, score=score)
        check_route(P, logits_of(70, E, dtype, k, kind), k, score=score, renormalize=False, bias=dev(np.zeros(E)))


def test_route_near_ties_are_decided_in_64_bits(P):
    """Scores that differ by less than fp32 shows: sigmoid(l) + b with b chosen so that two
    experts lie a few 2^-40 apart."""
    T, E = 64, 32
    g = rng(4)
    l = g.standard_normal((T, E)).astype(np.float32)
    l[:, 1::2] = l[:, ::2] + 0.5
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    l2 = np.repeat(l[:1], T, 0)
    s = np.repeat(s[:1], T, 0)
    b = np.zeros(E, np.float32)
    b[::2] = (s[0, 1::2] - s[0, ::2]).astype(np.float32)  # evens next to odds
    gap = np.abs(s[0, ::2] + b[::2].astype(np.float64) - s[0, 1::2])
    assert gap.max() < 2.0 ** -24 and gap.min() > 0
    check_route(P, dev(l2), 8, score="sigmoid", bias=dev(b))


def test_route_special_biases_and_shapes(P):
    E = 24
    l = logits_of(9, E, "f32", 5)
    b = np.zeros(E, np.float32)
    b[3], b[4], b[5] = np.inf, -np.inf, np.nan
    check_route(P, l, 24, score="sigmoid", bias=dev(b))
    # rows further apart than they are long, odd starts
    wide = logits_of(9, 101, "bf16", 6)
    check_route(P, wide[:, 3:60], 7)
    idx, w = P.route(wide[:0], 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    with pytest.raises(ValueError):
        P.route(wide.t(), 2)
    with pytest.raises(P.SparseFFNError):
        P.route(wide, 102)
    with pytest.raises(ValueError):
        P.route(wide.double(), 2)
    with pytest.raises(ValueError):
        P.route(wide, 2, score="tanh")


# --------------------------------------------------------------------------------- 8-bit rows
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,K", [(1, 1), (3, 2), (2, 15), (5, 16), (4, 17), (7, 255), (3, 1013), (2, 4096),
                                 (2, 11008), (1, 70001), (300, 64)])
def test_quantize_rows(P, dtype, R, K):
    say("quantize", dtype, R, K)
    x = dev(rng(5, R, K).standard_normal((R, K)) * 3, DT[dtype])
    q, s = P.quantize_rows(x)
    rq, rs = ref.quantize(f64(x))
    assert np.array_equal(f64(q), rq) and np.array_equal(f64(s), rs)
    if K % 16:  # room behind the rows is zero
        room = q.as_strided((R, q.stride(0) if R > 1 else (K + 15) // 16 * 16), (q.stride(0), 1))
        assert int(room[:, K:].abs().sum()) == 0


def test_quantize_borders(P):
    """Values on and next to the border between two whole numbers, for scales that are powers
    of two (the border is a 32-bit number) and scales that are not."""
    n = np.arange(-126, 127) + 0.5
    rows = []
    for amax in (127.0, 127.0 * 2 ** -20, 1.0, 3.3, 1e30, 7e-25):
        s = float(np.float32(amax) * (np.float32(1) / np.float32(127)))
        b = (n * s).astype(np.float32)
        rows.append(np.concatenate([[np.float32(amax)], b, np.nextafter(b, np.float32(np.inf)),
                                    np.nextafter(b, np.float32(-np.inf))]))
    x = dev(np.stack(rows))
    q, s = P.quantize_rows(x)
    rq, rs = ref.quantize(f64(x))
    assert np.array_equal(f64(s), rs) and np.array_equal(f64(q), rq)


def test_quantize_special_rows(P):
    x = np.zeros((9, 40), np.float32)
    x[1, 3] = np.nan
    x[2, 5] = np.inf
    x[3, 39] = -np.inf
    x[4] = 1e-45
    x[5, 7] = -2.0 ** -100
    x[6, 7] = 2.0 ** -101
    x[7] = 3.4e38
    x[8] = -0.0
    q, s = P.quantize_rows(dev(x))
    rq, rs = ref.quantize(x)
    assert np.array_equal(f64(s), rs, equal_nan=True) and np.array_equal(f64(q), rq)
    assert math.isnan(float(s[1])) and float(s[4]) == 0 and int(q[5, 7]) == -127
    # strides: a transposed matrix is copied, columns of a wider one are read in place
    y = dev(rng(6).standard_normal((33, 50)))
    for v in (y.t(), y[:, 7:30], y.reshape(3, 11, 50)):
        q, s = P.quantize_rows(v)
        rq, rs = ref.quantize(f64(v).reshape(-1, v.shape[-1]))
        assert np.array_equal(f64(q).reshape(rq.shape), rq)
        assert np.array_equal(f64(s).reshape(-1), rs)
    q, s = P.quantize_rows(y[:0])
    assert q.shape == (0, 50) and s.shape == (0,)


# ---------------------------------------------------------------------------------- products
def weights_of(P, *shape, seed=0):
    return P.quantize_rows(dev(rng(7, seed, *shape).standard_normal(shape) * 0.02))


def check_matmul(P, M, K, N, xt, yt, bias, seed=0):
    g = rng(8, M, K, N, seed)
    w, ws = weights_of(P, N, K, seed=seed)
    b = dev(g.standard_normal(N)) if bias else None
    x = dev(g.standard_normal((M, K)) * 2, DT.get(xt, torch.float32))
    if xt == "i8":
        x, xs = P.quantize_rows(x)
        y = P.i8_matmul(x, w, ws, x_scale=xs, bias=b, out_dtype=DT[yt])
        q, s = f64(x), f64(xs)
    else:
        y = P.i8_matmul(x, w, ws, bias=b, out_dtype=DT[yt])
        q, s = ref.quantize(f64(x))
    want, mag = ref.matmul(q, s, f64(w), f64(ws), None if b is None else f64(b))
    assert y.dtype == DT[yt] and y.shape == (M, N)
    check(y, want, 4 * U * mag, DT[yt])


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("K,N", [(1, 1), (16, 16), (17, 3), (127, 65), (128, 64), (129, 130), (1013, 1101),
                                 (4096, 520), (2064, 257)])
def test_matmul_sizes(P, M, K, N):
    say("matmul", M, K, N)
    for i, (xt, yt) in enumerate((("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("i8", "f32"))):
        check_matmul(P, M, K, N, xt, yt, (M + i) % 2 == 0)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 11008), (3, 11008, 4096), (24, 11008, 4096), (700, 4096, 2049),
                                   (513, 192, 4104)])
@pytest.mark.parametrize("xt,yt", [("f16", "f32"), ("i8", "bf16")])
def test_matmul_large(P, M, K, N, xt, yt):
    say("matmul", M, K, N, xt, yt)
    check_matmul(P, M, K, N, xt, yt, True)


@pytest.mark.parametrize("M,K", [(1, 65536), (1, 65537), (2, 32768), (3, 20000), (4, 16384), (4, 16385), (5, 300)])
def test_matmul_around_what_lds_holds(P, M, K):
    """Rows that the product holds in 8 bits itself, up to the most it takes, and just above."""
    say("matmul lds", M, K)
    for xt in ("f32", "bf16"):
        check_matmul(P, M, K, 40, xt, "f32", True)


@pytest.mark.parametrize("k,f", [(1, 65536), (2, 32768), (2, 32769), (4, 16384), (16, 4096), (17, 300), (64, 1024)])
def test_experts_one_token_around_what_lds_holds(P, k, f):
    say("experts lds", k, f)
    E = min(k, 5)
    ffn = make_experts(P, E, 48, f, True, False)
    idx, w = tables(1, E, k, dropped=0.3)
    x = dev(rng(37, k, f).standard_normal((1, 48)), torch.float16)
    check_experts(P, ffn, x, idx, w, torch.float32)


def test_matmul_extreme_values(P):
    """Every product at its largest: the sums stay in 32 bits up to the longest row."""
    K = 131071
    for M in (1, 40):
        x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        w = torch.full((5, (K + 15) // 16 * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
        w[1] = 127
        one = torch.ones(5, device="cuda")
        y = P.i8_matmul(x, w, one, x_scale=torch.ones(M, device="cuda"))
        want = np.array([16384.0 * K, -128.0 * 127 * K] + [16384.0 * K] * 3)
        assert (np.abs(f64(y) - want) <= U * np.abs(want)).all()


@pytest.mark.parametrize("M,K,N", [(4100, 48, 7931), (4099, 40, 7934), (1100, 80, 14597), (200, 33, 16389),
                                   (65, 70, 1013)])
@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
def test_matmul_tiles_write_only_their_rows(P, M, K, N, yt):
    """Each of the tiles of many rows, rows and channels that end inside one, a window of a
    larger output at an odd column."""
    say("matmul tiles", M, K, N, yt)
    w, ws = weights_of(P, N, K)
    x, xs = P.quantize_rows(dev(rng(38, M, K).standard_normal((M, K))))
    b = dev(rng(39, N).standard_normal(N))
    out = torch.full((M + 2, N + 9), -7.0, dtype=DT[yt], device="cuda")
    P.i8_matmul(x, w, ws, x_scale=xs, bias=b, y=out[1:-1, 3:3 + N])
    want, mag = ref.matmul(f64(x), f64(xs), f64(w), f64(ws), f64(b))
    check(out[1:-1, 3:3 + N], want, 4 * U * mag, DT[yt])
    out[1:-1, 3:3 + N] = -7.0
    assert (out == -7.0).all()


def test_matmul_strides_and_untouched_memory(P):
    M, K, N = 37, 200, 77
    g = rng(9)
    wide = dev(g.standard_normal((M, 331)))
    room = torch.full((N + 2, 240), 99, dtype=torch.int8, device="cuda")  # garbage behind the rows
    q, ws = weights_of(P, N, K)
    room[1:-1, :K] = q
    w = room[1:-1, :K]
    out = torch.full((M + 2, 90), -7.0, dtype=torch.float16, device="cuda")
    x = wide[:, 5:5 + K]
    P.i8_matmul(x, w, ws, y=out[1:-1, 3:3 + N])
    rq, rs = ref.quantize(f64(x))
    want, mag = ref.matmul(rq, rs, f64(q), f64(ws))
    check(out[1:-1, 3:3 + N], want, 4 * U * mag, torch.float16)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:-1, 3:3 + N] = False
    assert bool((out[keep] == -7.0).all())
    # int8 rows at odd places, garbage behind their ends
    xi = torch.full((M, 301), 77, dtype=torch.int8, device="cuda")
    xi[:, 3:3 + K] = dev(rq, torch.int8)
    y = P.i8_matmul(xi[:, 3:3 + K], w, ws, x_scale=dev(rs))
    check(y, want, 4 * U * mag, torch.float32)


def test_matmul_rows_that_are_not_finite_or_zero(P):
    K, N = 96, 40
    for M in (6, 70):
        x = rng(10, M).standard_normal((M, K)).astype(np.float32)
        x[1, 4], x[2, 5], x[3] = np.nan, -np.inf, 0.0
        w, ws = weights_of(P, N, K)
        b = dev(rng(11).standard_normal(N))
        y = f64(P.i8_matmul(dev(x), w, ws, bias=b))
        assert np.isnan(y[1:3]).all() and np.isfinite(np.delete(y, (1, 2), 0)).all()
        assert np.array_equal(y[3], f64(b))


def test_matmul_refusals(P):
    w, ws = weights_of(P, 8, 32)
    x = dev(rng(12).standard_normal((3, 32)))
    for bad in (dict(x_scale=ws[:3]), dict(bias=ws.double()), dict(bias=ws[:7]), dict(out_dtype=torch.float64),
                dict(y=torch.empty((3, 7), device="cuda")), dict(work=torch.empty(9, device="cuda")),
                dict(bias=ws.cpu())):
        with pytest.raises(ValueError):
            P.i8_matmul(x, w, ws, **bad)
    with pytest.raises(ValueError):  # int8 rows without scales
        P.i8_matmul(torch.zeros((3, 32), dtype=torch.int8, device="cuda"), w, ws)
    with pytest.raises(ValueError):  # rows on odd places
        P.i8_matmul(x[:, :31], torch.zeros((8, 31), dtype=torch.int8, device="cuda"), ws)
    with pytest.raises(ValueError):  # no room behind the last row
        P.i8_matmul(x[:, :30], torch.zeros(8 * 32 - 2, dtype=torch.int8, device="cuda").as_strided((8, 30), (32, 1)), ws)
    with pytest.raises(P.SparseFFNError):  # scratch too small
        P.i8_matmul(x.repeat(3, 1), w, ws, work=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert P.i8_matmul(x[:0], w, ws).shape == (0, 8)


def test_matmul_offsets_past_32_bits(P):
    """More than 2^31 outputs: the last rows against the reference."""
    M, K, N = 200_003, 64, 11008
    w, ws = weights_of(P, N, K)
    x = torch.randn((M, K), device="cuda", dtype=torch.bfloat16)
    y = P.i8_matmul(x, w, ws)
    pick = torch.tensor([0, 97_541, 195_083, 195_084, M - 2, M - 1], device="cuda")
    rq, rs = ref.quantize(f64(x[pick]))
    want, mag = ref.matmul(rq, rs, f64(w), f64(ws))
    check(y[pick], want, 4 * U * mag, torch.bfloat16)


# ----------------------------------------------------------------------------------- experts
def make_experts(P, E, d, f, gated, bias, seed=0):
    g = rng(13, E, d, f, seed)
    m = [dev(g.standard_normal((E, f, d)) * 0.05) for _ in range(2 if gated else 1)]
    down = dev(g.standard_normal((E, d, f)) * 0.05)
    b = dev(g.standard_normal((E, f)) * 0.3) if bias else None
    return P.ExpertFFN.from_float(w_act=m[0], w_up=m[1] if gated else None, w_down=down, b_act=b)


def tables(T, E, k, seed=0, dropped=0.2):
    g = rng(14, T, E, k, seed)
    idx = g.integers(0, E, (T, k)).astype(np.int32)
    idx[g.random((T, k)) < dropped] = -1
    return dev(idx, torch.int32), dev(g.random((T, k)))


def check_experts(P, ffn, x, idx, w, yt, y=None):
    y = ffn(x, idx, w, out_dtype=yt) if y is None else y
    k = idx.shape[1]
    want, mag = ref.experts(f64(x), to_np(idx), to_np(w), to_np(ffn.w_act), to_np(ffn.act_scale),
                            to_np(ffn.w_down), to_np(ffn.down_scale),
                            None if ffn.b_act is None else to_np(ffn.b_act))
    check(y, want, (k + 4) * U * mag, yt)
    return y


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 40, 150])
@pytest.mark.parametrize("E,k,d,f", [(1, 1, 16, 16), (2, 2, 1, 1), (3, 1, 130, 65), (4, 2, 128, 256),
                                     (8, 3, 200, 333), (64, 6, 64, 100), (5, 5, 1025, 190)])
@pytest.mark.parametrize("gated", [True, False])
def test_experts_sizes(P, T, E, k, d, f, gated):
    say("experts", T, E, k, d, f, gated)
    ffn = make_experts(P, E, d, f, gated, bias=T % 2 == 0)
    idx, w = tables(T, E, k)
    for i, (xt, yt) in enumerate((("f32", "f32"), ("f16", "bf16"), ("bf16", "f16"))):
        x = dev(rng(15, T, d, i).standard_normal((T, d)), DT[xt])
        check_experts(P, ffn, x, idx, w, DT[yt])


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (16, 4, 2), (600, 4, 2), (300, 1, 1)])
def test_experts_larger(P, T, E, k):
    say("experts larger", T, E, k)
    ffn = make_experts(P, E, 1024, 1408, True, False)
    idx, w = tables(T, E, k, dropped=0.0)
    x = dev(rng(16, T).standard_normal((T, 1024)), torch.bfloat16)
    y = ffn(x, idx, w)
    pick = sorted(set([0, T - 1] + list(rng(17).integers(0, T, 12))))
    check_experts(P, ffn, x[pick], idx[pick], w[pick], torch.bfloat16, y=y[pick])


def test_experts_all_on_one_and_none(P):
    """Every token to the last expert, one expert twice in a token, tokens without any."""
    ffn = make_experts(P, 6, 96, 160, True, True)
    T = 210
    x = dev(rng(18).standard_normal((T, 96)))
    idx = torch.full((T, 3), -1, dtype=torch.int32, device="cuda")
    idx[:, 0] = 5
    idx[5, 1] = 5
    idx[7], idx[8] = -1, 6  # none; past the last expert
    idx[9] = torch.tensor([-2147483648, 2147483647, 2], dtype=torch.int32)
    w = dev(rng(19).random((T, 3)))
    w[7], w[8] = math.nan, math.inf  # weights of slots without an expert are not read
    y = check_experts(P, ffn, x, idx, w, torch.float32)
    assert bool((y[7:9] == 0).all())
    none = torch.full((T, 3), -1, dtype=torch.int32, device="cuda")
    assert bool((ffn(x, none, w) == 0).all())


@pytest.mark.parametrize("gated", [True, False])
def test_experts_nan_stays_in_its_token(P, gated):
    ffn = make_experts(P, 3, 64, 48, gated, False)
    for T in (4, 90):
        x = rng(20, T).standard_normal((T, 64)).astype(np.float32)
        x[1, 3], x[2, 4] = np.nan, np.inf
        idx, w = tables(T, 3, 2, dropped=0.0)
        y = f64(ffn(dev(x), idx, w))
        assert np.isnan(y[1:3]).all()
        assert np.isfinite(np.delete(y, (1, 2), 0)).all()


def test_experts_activation_overflow_is_nan(P):
    """h beyond fp32 makes its token NaN, not a wrong number."""
    ffn = make_experts(P, 2, 64, 48, True, False)
    x = dev(rng(21).standard_normal((3, 64)))
    x[1] *= 1e25
    idx, w = tables(3, 2, 2, dropped=0.0)
    y = f64(ffn(x, idx, w))
    assert np.isnan(y[1]).all() and np.isfinite(y[[0, 2]]).all()


def test_experts_strides_chunks_and_untouched_memory(P):
    ffn = make_experts(P, 4, 100, 72, True, True)
    T, k = 93, 2
    wide = dev(rng(22).standard_normal((T, 151)))
    x = wide[:, 9:109]
    idx, w = tables(T, 4, k)
    out = torch.full((T + 2, 120), 5.0, device="cuda")
    ffn(x, idx, w, y=out[1:-1, 4:104])
    check_experts(P, ffn, x, idx, w, torch.float32, y=out[1:-1, 4:104])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:-1, 4:104] = False
    assert bool((out[keep] == 5.0).all())
    for tokens in (1, 7, 50):  # scratch for fewer tokens: in chunks, the same values
        y = ffn(x, idx, w, work=ffn.work(tokens, k))
        assert torch.equal(y, out[1:-1, 4:104])
    y2 = P.experts(x, idx, w, ffn.w_act, ffn.act_scale, ffn.w_down, ffn.down_scale, b_act=ffn.b_act)
    assert torch.equal(y2, y)


def test_experts_weights_with_room_and_dense(P):
    """Rows with garbage behind them; one expert as a dense FFN."""
    ffn = make_experts(P, 1, 50, 70, False, False)
    wa = torch.full((1, 70, 96), 111, dtype=torch.int8, device="cuda")
    wa[..., :50] = ffn.w_act
    wd = torch.full((1, 50, 80), -111, dtype=torch.int8, device="cuda")
    wd[..., :70] = ffn.w_down
    other = P.ExpertFFN(w_act=wa[..., :50], act_scale=ffn.act_scale, w_down=wd[..., :70],
                        down_scale=ffn.down_scale)
    x = dev(rng(23).standard_normal((20, 50)))
    y = ffn.dense(x)
    assert torch.equal(y, other.dense(x))
    one = torch.ones((20, 1), device="cuda")
    check_experts(P, ffn, x, torch.zeros((20, 1), dtype=torch.int32, device="cuda"), one, torch.float32, y=y)
    with pytest.raises(ValueError):
        make_experts(P, 2, 50, 70, False, False).dense(x)


def test_experts_refusals(P):
    ffn = make_experts(P, 4, 64, 48, True, False)
    x = dev(rng(24).standard_normal((5, 64)))
    idx, w = tables(5, 4, 2)
    for args in ((x[:, :63], idx, w), (x, idx.long(), w), (x, idx[:4], w), (x, idx, w.half()),
                 (x, idx, w[:, :1]), (x.t().contiguous().t(), idx, w), (x, idx.cpu(), w), (x.double(), idx, w)):
        with pytest.raises(ValueError):
            ffn(*args)
    with pytest.raises(P.SparseFFNError):
        ffn(x, idx, w, work=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(P.SparseFFNError):
        ffn(x, torch.zeros((5, 65), dtype=torch.int32, device="cuda"), torch.zeros((5, 65), device="cuda"))
    with pytest.raises(ValueError):
        P.ExpertFFN(w_act=ffn.w_act, act_scale=ffn.act_scale, w_down=ffn.w_down[:, :, :47],
                    down_scale=ffn.down_scale)
    assert ffn(x[:0], idx[:0], w[:0]).shape == (0, 64)


def test_matmul_activations_past_32_bits(P):
    """int8 rows in place, 4.7 GB of them."""
    M, K, N = 36_000, 131_072 - 128, 8
    x = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    g = rng(35)
    pick = [0, 5000, 32_767, 32_768, 32_769, 35_999]
    rows = g.integers(-127, 128, (len(pick), K)).astype(np.int8)
    x[pick] = torch.from_numpy(rows).to("cuda")
    w = torch.from_numpy(g.integers(-127, 128, (N, K)).astype(np.int8)).to("cuda")
    ws, xs = torch.rand(N, device="cuda"), torch.rand(M, device="cuda")
    y = P.i8_matmul(x, w, ws, x_scale=xs)
    want, mag = ref.matmul(rows, f64(xs[pick]), f64(w), f64(ws))
    check(y[pick], want, 4 * U * mag, torch.float32)
    assert int((y != 0).any(1).sum()) == len(pick)


def test_experts_many_slots(P):
    """More slots than the sort keeps in registers, very uneven, several thousand dropped."""
    T, E, k = 6001, 9, 3
    ffn = make_experts(P, E, 32, 48, True, False)
    g = rng(36)
    idx = np.minimum(g.geometric(0.5, (T, k)) - 1, E).astype(np.int32)  # E: no expert
    idx[g.random((T, k)) < 0.15] = -1
    idx, w = dev(idx, torch.int32), dev(g.random((T, k)))
    x = dev(g.standard_normal((T, 32)))
    check_experts(P, ffn, x, idx, w, torch.float32)


def test_experts_offsets_past_32_bits(P):
    """More than 2^31 bytes of weights: the last expert against the reference."""
    E, d, f = 26, 4096, 11008
    wa = torch.zeros((E, f, 2, d), dtype=torch.int8, device="cuda")
    wd = torch.zeros((E, d, f), dtype=torch.int8, device="cuda")
    small = make_experts(P, 1, d, f, True, False)
    wa[-1], wd[-1] = small.w_act[0], small.w_down[0]
    sa, sd = small.act_scale.expand(E, f, 2).contiguous(), small.down_scale.expand(E, d).contiguous()
    for T in (1, 70):
        x = dev(rng(25, T).standard_normal((T, d)))
        idx = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
        one = torch.ones((T, 1), device="cuda")
        y = P.experts(x, idx, one, wa, sa, wd, sd)
        assert torch.equal(y, small.dense(x))
        check_experts(P, small, x[:2], idx[:2] * 0, one[:2], torch.float32, y=y[:2])


# ---------------------------------------------------------------------- together, graphs, streams
def layer(P, x, wr, ffn, k):
    logits = x.float() @ wr
    idx, w = P.route(logits, k, score="sigmoid", groups=4, top_groups=2, scale=1.5)
    return logits, idx, w, ffn(x, idx, w)


@pytest.mark.parametrize("T", [1, 9, 200])
def test_layer_of_experts(P, T):
    """A router's logits, the choice, the experts: a mixture-of-experts layer as it is used,
    against the 64-bit forms chained (from the logits on)."""
    E, d, f, k = 16, 192, 320, 4
    ffn = make_experts(P, E, d, f, True, False)
    wr = dev(rng(26).standard_normal((d, E)) * 0.1)
    x = dev(rng(27, T).standard_normal((T, d)), torch.bfloat16)
    logits, idx, w, y = layer(P, x, wr, ffn, k)
    ri, rw = ref.route(f64(logits), k, score="sigmoid", groups=4, top_groups=2, scale=1.5)
    assert np.array_equal(to_np(idx), ri)
    check_experts(P, ffn, x, idx, w, torch.bfloat16, y=y)


def test_layer_with_an_8_bit_projection_in_front(P):
    """An 8-bit product whose bf16 output feeds the router and the experts."""
    E, d, f, k, T = 8, 256, 128, 2, 33
    ffn = make_experts(P, E, d, f, False, True)
    w, ws = weights_of(P, d, 144, seed=3)
    wr = dev(rng(28).standard_normal((d, E)))
    x0 = dev(rng(29).standard_normal((T, 144)), torch.bfloat16)
    x = P.i8_matmul(x0, w, ws)
    logits, idx, wt, y = layer(P, x, wr, ffn, k)
    rq, rs = ref.quantize(f64(x0))
    want, mag = ref.matmul(rq, rs, f64(w), f64(ws))
    check(x, want, 4 * U * mag, torch.bfloat16)
    check_experts(P, ffn, x, idx, wt, torch.bfloat16, y=y)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_graph_replays(P, T):
    """Two captured layers of different sizes (scratch of their own), replayed in turn with
    eager work between, on new inputs each time."""
    k = 2
    sets = []
    for j, (E, d, f) in enumerate(((8, 128, 192), (4, 256, 100))):
        ffn = make_experts(P, E, d, f, True, False, seed=j)
        w, ws = weights_of(P, 72, d, seed=j)
        x = torch.zeros((T, d), device="cuda", dtype=torch.float16)
        l = torch.zeros((T, E), device="cuda")

        def run(x=x, l=l, ffn=ffn, w=w, ws=ws):
            idx, wt = P.route(l, k)
            y = ffn(x, idx, wt)
            return idx, wt, y, P.i8_matmul(y, w, ws)

        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        sets.append((x, l, run, g, out))
    for it in range(5):
        for j, (x, l, run, g, out) in enumerate(sets):
            x.copy_(dev(rng(30, it, j).standard_normal(x.shape), torch.float16))
            l.copy_(dev(rng(31, it, j).standard_normal(l.shape)))
            g.replay()
        for x, l, run, g, out in sets:
            want = run()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_another_stream(P):
    ffn = make_experts(P, 4, 128, 192, True, False)
    idx, w = tables(50, 4, 2)
    x = dev(rng(32).standard_normal((50, 128)))
    l = dev(rng(33).standard_normal((50, 4)))
    one = make_experts(P, 1, 128, 192, True, False)
    want = (ffn(x, idx, w), *P.route(l, 2), *P.quantize_rows(x), one.dense(x))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = (ffn(x, idx, w, stream=s), *P.route(l, 2, stream=s), *P.quantize_rows(x, stream=s),
               one.dense(x, stream=s))
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_another_stream_takes_no_memory_that_this_one_still_uses(P):
    """A tensor that is freed here while a queued copy still reads it: a call on another stream
    that does not wait for this one must not get its memory."""
    ffn = make_experts(P, 2, 1024, 64, True, False)
    idx, w = tables(512, 2, 1, dropped=0.0)
    x = dev(rng(38).standard_normal((512, 1024)))
    l = dev(rng(39).standard_normal((512, 2)))
    s = torch.cuda.Stream()
    want = ffn(x, idx, w)
    torch.cuda.synchronize()
    for _ in range(3):
        a = torch.full((512, 1024), 3.0, device="cuda")
        a2 = torch.full((512, 1), 7, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        b, b2 = a.clone(), a2.clone()
        del a, a2
        y = ffn(x, idx, w, stream=s)
        P.route(l, 1, stream=s)
        s.synchronize()
        torch.cuda.synchronize()
        assert bool((b == 3.0).all()) and bool((b2 == 7).all())
        assert torch.equal(y, want)


def test_output_over_the_input(P):
    ffn = make_experts(P, 3, 128, 96, True, False)
    for T in (1, 5, 100):
        idx, w = tables(T, 3, 2)
        x = dev(rng(40, T).standard_normal((T, 128)))
        want = ffn(x, idx, w)
        x2 = x.clone()
        ffn(x2, idx, w, y=x2)
        assert torch.equal(x2, want)


def test_same_values_every_time(P):
    ffn = make_experts(P, 8, 512, 700, True, False)
    for T in (3, 500):
        idx, w = tables(T, 8, 3)
        x = dev(rng(34, T).standard_normal((T, 512)))
        first = ffn(x, idx, w)
        for _ in range(4):
            assert torch.equal(ffn(x, idx, w), first)
