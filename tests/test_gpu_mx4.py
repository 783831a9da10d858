"""GPU tests of rows in 4-bit blocks and their products (quantize_mx4, dequantize_mx4, mx4_matmul)
against plain 64-bit forms (tests/mx4_ref.py): lengths from one to long, every type, borders between
two codes and between two scales, the smallest and largest scales, NaN, strides, other streams,
graph replays.

Tolerances, each from the roundings made (u = 2^-24, half a step of fp32):
 - codes, scales and fp32 values of blocks are equal; 16-bit values are the fp32 ones rounded;
 - products: a matrix instruction adds the exact products of 128 columns to a 32-bit sum, cutting
   what lies below the sum's last places: at most 2 steps (4 u) of the magnitudes that it adds.
   ceil(K / 128) of them, a few additions of partial sums and the bias: (4 ceil(K / 128) + 16) u
   sum |x w|, then half a step of the output type. Results below 2^-126 may be off by 2^-126.
   Sums are held in 32 bits: every partial sum is at most sum |x w|, so where that is below 2^127
   none passes the largest 32-bit number (2^128 (1 - u)) and the bound holds; where it is not, a
   partial sum may be infinite, and nothing is asked."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import mx4_sizes
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


def roomy(q, E, spare=0):
    """Packed rows on the device with room behind the scales (filled with `spare`)."""
    R, B = E.shape
    room = np.full((R, (B + 15) // 16 * 16), spare, np.uint8)
    room[:, :B] = E
    return dev(q, torch.uint8), dev(room, torch.uint8)[:, :B]


def check_blocks(P, x):
    q, s = P.quantize_mx4(x)
    code, E = ref.blocks(f64(x))
    rq, rE = ref.pack(code, E)
    assert np.array_equal(to_np(s), rE)
    assert np.array_equal(to_np(q), rq)
    K = x.shape[1]
    want = torch.from_numpy(ref.values(rq, rE)[:, :K]).float()
    for dt in DT.values():
        y = P.dequantize_mx4(q, s, cols=K, dtype=dt).cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        w = want.to(dt)
        assert torch.equal(torch.nan_to_num(y, 0.0, 1.0, -1.0), torch.nan_to_num(w, 0.0, 1.0, -1.0))
    return q, s


@pytest.mark.parametrize("K", [1, 2, 7, 8, 31, 32, 33, 63, 64, 96, 511, 512, 513, 1013, 4096, 4100, 70001])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_blocks_sizes(P, K, dtype):
    say("blocks", K, dtype)
    for R in (1, 3, 130 if K < 5000 else 2):
        g = rng(1, K, R)
        check_blocks(P, dev(g.standard_normal((R, K)) * 2.0 ** g.integers(-8, 8, (R, 1)), DT[dtype]))


def test_blocks_borders(P):
    """Every border between two codes, and the numbers next to it, at many scales; and every border
    between two scales."""
    say("blocks borders")
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 2.0, 3.0, 4.0], np.float32)
    near = np.concatenate([mid, np.nextafter(mid, np.float32(9)), np.nextafter(mid, np.float32(-9))])
    rows = []
    for e in (-126, -120, -40, -1, 0, 1, 30, 100, 124):
        for block in np.array_split(near, 2):
            r = np.zeros(32)
            r[:len(block)] = block.astype(np.float64)
            r[len(block)] = -6.5
            rows.append(r * 2.0 ** e)
    for e in (-126, -60, 0, 60, 125):
        for top in (3.5, 7.0, 4.0, 6.0, 1.75):
            t = np.float32(top * 2.0 ** min(e, 125 if top < 4 else 124))
            for v in (t, np.nextafter(t, np.float32(0)), np.nextafter(t, np.float32(np.inf))):
                r = np.zeros(32)
                r[5], r[6], r[7] = -v, v / 2, v / 16
                rows.append(r)
    x = np.array(rows, np.float32)
    assert np.isfinite(x).all()
    check_blocks(P, dev(x))


def test_blocks_far(P):
    """Zeros of either sign, subnormal numbers, the largest ones, infinities and NaN, each in blocks
    beside ordinary ones."""
    say("blocks far")
    g = rng(2)
    x = g.standard_normal((40, 128)).astype(np.float32)
    x[0] = 0.0
    x[1, :64] = -0.0
    x[2, 40:44] = [np.nan, 1e30, -1e30, 0]
    x[3, 32] = np.inf
    x[4, 127] = -np.inf
    x[5] = 2.0 ** -149
    x[6] = g.standard_normal(128) * 2.0 ** -130
    x[7] = g.standard_normal(128) * 2.0 ** -124
    x[8, :32] = np.finfo(np.float32).max
    x[9] = g.standard_normal(128) * 2.0 ** 120
    x[10, ::2] = 2.0 ** -149
    check_blocks(P, dev(x))
    check_blocks(P, dev(x[:8], torch.bfloat16))
    h = (x[:8].clip(-6e4, 6e4) * 2.0 ** -20).astype(np.float16)
    check_blocks(P, dev(h, torch.float16))


def test_blocks_strides_and_shapes(P):
    say("blocks strides")
    g = rng(3)
    big = dev(g.standard_normal((20, 333)))
    for x in (big[:, 5:104], big[::3, 1:66], big[4:5, :65], big[:, :1], big.t()[:40].t().contiguous().t().t()):
        check_blocks(P, x)
    x3 = dev(g.standard_normal((3, 4, 70)))
    q, s = P.quantize_mx4(x3)
    assert q.shape == (3, 4, 48) and s.shape == (3, 4, 3)
    q2, s2 = P.quantize_mx4(x3.view(12, 70))
    assert torch.equal(q.view(12, 48), q2) and torch.equal(s.reshape(12, 3), s2)
    y = P.dequantize_mx4(q, s, cols=70)
    assert torch.equal(y.view(12, 70), P.dequantize_mx4(q2, s2, cols=70))
    q1, s1 = P.quantize_mx4(x3[0, 0])
    assert torch.equal(q1, q[0, 0]) and torch.equal(P.dequantize_mx4(q1, s1)[:70], y[0, 0])
    t = x3.transpose(0, 1)  # no view as a matrix: copied
    qt, st = P.quantize_mx4(t)
    assert torch.equal(qt, q.transpose(0, 1)) and torch.equal(st, s.transpose(0, 1))
    e, se = P.quantize_mx4(dev(np.zeros((0, 40))))
    assert e.shape == (0, 32) and P.dequantize_mx4(e, se, cols=40).shape == (0, 40)
    with pytest.raises(ValueError):
        P.dequantize_mx4(q2, s2, cols=97)
    with pytest.raises(ValueError):
        P.dequantize_mx4(q2, s2, cols=64)
    with pytest.raises(ValueError):
        P.dequantize_mx4(q2, s2.contiguous())  # rows of scales that begin anywhere


def test_blocks_leave_the_rest(P):
    """What lies between the rows of codes, scales and values stays as it was."""
    say("blocks leave the rest")
    N = P._native
    x = dev(rng(4).standard_normal((5, 70)))
    q = torch.full((5, 80), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((5, 16), 99, dtype=torch.uint8, device="cuda")
    N.sparse_ffn_quantize_mx4(x.data_ptr(), 0, 70, 5, 70, q.data_ptr(), 80, s.data_ptr(), 16, 0)
    torch.cuda.synchronize()
    rq, rs = P.quantize_mx4(x)
    assert torch.equal(q[:, :48], rq) and (q[:, 48:] == 77).all()
    assert torch.equal(s[:, :3], rs) and (s[:, 3:] == 99).all()
    y = torch.full((5, 75), 3.0, device="cuda")
    N.sparse_ffn_dequantize_mx4(q.data_ptr(), 80, s.data_ptr(), 16, 5, 70, y.data_ptr(), 0, 75, 0)
    torch.cuda.synchronize()
    assert torch.equal(y[:, :70], P.dequantize_mx4(rq, rs, cols=70)) and (y[:, 70:] == 3.0).all()


@pytest.mark.parametrize("cols", [0, -1, -33, 97])
def test_columns_that_no_blocks_hold(P, cols):
    say("columns", cols)
    q, s = P.quantize_mx4(dev(rng(5).standard_normal((2, 70))))
    with pytest.raises(ValueError):
        P.dequantize_mx4(q, s, cols=cols)
    with pytest.raises(ValueError):
        P.dequantize_mx4(q[:1, :16], s[:1, :1], cols=cols)


def test_blocks_of_many_long_rows(P):
    """More rows than one launch has workgroups for beside the pieces of long rows."""
    say("many long rows")
    R, K = (1 << 14) + 33, 131100
    x = torch.randn((R, K), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    q, s = P.quantize_mx4(x)
    y = P.dequantize_mx4(q, s, cols=K)
    for r in (0, 8000, R - 40):
        rows = slice(r, r + 40)
        rq, rs = P.quantize_mx4(x[rows])
        assert torch.equal(q[rows], rq) and torch.equal(s[rows], rs)
        assert torch.equal(y[rows], P.dequantize_mx4(rq, rs, cols=K))


def test_slices_of_many_rows_on_another_stream(P):
    """Codes whose rows lie the same distance apart are read where they are, also on a stream that does
    not wait for this one's work; others are refused, as their scales are."""
    say("slices on another stream")
    x = dev(rng(6).standard_normal((4, 6, 70)))
    q, s = P.quantize_mx4(x)
    want = P.dequantize_mx4(q, s, cols=70)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    y = P.dequantize_mx4(q[:, ::2], s[:, ::2], cols=70, stream=other)
    z = P.dequantize_mx4(q[1:, 3], s[1:, 3], cols=70, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(y, want[:, ::2]) and torch.equal(z, want[1:, 3])
    with pytest.raises(ValueError):
        P.dequantize_mx4(q[:, :2], s[:, :2], cols=70)


# --------------------------------------------------------------------------------- products
def check_product(got, x, w, bias, dtype):
    """x, w: 64-bit values of the rows in blocks."""
    want, mag = ref.matmul(x, w, bias)
    got = f64(got)
    bad = np.isnan(mag)  # a NaN block reaches these
    assert np.isnan(got[bad]).all()
    with np.errstate(invalid="ignore"):
        err = (4 * ((x.shape[1] + 127) // 128) + 16) * U * mag + 2.0 ** -126
        fi = torch.finfo(dtype)
        lim = err + fi.eps / 2 * np.maximum(np.abs(want) + err, fi.tiny)
        d = np.abs(got - want)
        use = ~bad & (mag < 2.0 ** 127)
    off = int((~(d <= lim) & use).sum())
    assert off == 0, f"{off} values off, worst {np.max((d / lim)[use]):.3g} of the bound"


def held(x):
    """The values that 64-bit rows are held as."""
    code, E = ref.blocks(x)
    return ref.values(*ref.pack(code, E)), code, E


def problem(M, K, N, seed, spread=3):
    g = rng(5, M, K, N, seed)
    x = g.standard_normal((M, K)) * 2.0 ** g.integers(-spread, spread + 1, (M, 1))
    w = g.standard_normal((N, K)) * 2.0 ** g.integers(-spread, spread + 1, (N, 1))
    return x, w, g.standard_normal(N)


SIZES = [(1, 1, 1), (1, 32, 16), (1, 33, 17), (2, 64, 15), (3, 512, 100), (4, 1000, 64), (5, 544, 33),
         (7, 4096, 129), (16, 480, 257), (17, 129, 31), (31, 96, 70), (32, 2048, 500), (33, 700, 65),
         (48, 1536, 300), (64, 512, 128), (65, 513, 127), (100, 1013, 1101), (128, 256, 256),
         (130, 1024, 513), (200, 352, 700), (257, 1056, 300), (333, 160, 1030)]


@pytest.mark.parametrize("M,K,N", SIZES)
def test_product_sizes(P, M, K, N):
    say("product", M, K, N)
    x, w, b = problem(M, K, N, 0)
    wv, wc, wE = held(w)
    wq, ws = roomy(*ref.pack(wc, wE), spare=255)  # NaN scales behind the rows: without effect
    for i, (dt, out) in enumerate((("f32", "f32"), ("f16", "bf16"), ("bf16", "f16"))):
        xt = dev(x, DT[dt])
        xv, xc, xE = held(f64(xt))
        bias = b if i != 1 else None
        y = P.mx4_matmul(xt, wq, ws, bias=None if bias is None else dev(bias), out_dtype=DT[out])
        bf = None if bias is None else bias.astype(np.float32)
        check_product(y, xv, wv, bf, DT[out])
        # the same rows given in blocks: the same bits
        xq, xs = roomy(*ref.pack(xc, xE), spare=255)
        y2 = P.mx4_matmul(xq, wq, ws, x_scale=xs, bias=None if bias is None else dev(bias),
                          out_dtype=DT[out])
        assert torch.equal(y, y2)


@pytest.mark.parametrize("M,K,N", [(5, 1, 1), (5, 31, 4099), (9, 512, 8), (15, 33, 130), (16, 511, 9),
                                   (17, 512, 257), (18, 2, 16), (24, 78, 510), (40, 129, 3001),
                                   (250, 384, 1000), (4000, 65, 33), (1030, 511, 1011), (65000, 7, 2)])
def test_product_short_rows(P, M, K, N):
    """Rows of one group, a wave a tile: tiles with a few rows or channels, many of either."""
    test_product_sizes(P, M, K, N)


@pytest.mark.parametrize("M", [3, 5, 21, 300])
def test_product_short_rows_between(P, M):
    """Short rows of x, w, their scales and y further apart than they are long, at odd places, NaN and any
    codes between them; two graphs replayed in turn, on inputs and a bias that change."""
    say("product short strides", M)
    x, w, b = problem(M, 300, 75, 9)
    wv, wc, wE = held(w)
    pq, pE = ref.pack(wc, wE)
    wq = torch.full((75, 400), 0x77, dtype=torch.uint8, device="cuda")
    ws = torch.full((75, 48), 255, dtype=torch.uint8, device="cuda")
    wq[:, :160], ws[:, :10] = dev(pq, torch.uint8), dev(pE, torch.uint8)
    graphs = []
    for dt in (torch.float32, torch.float16):
        big = torch.full((M, 777), float("nan"), device="cuda", dtype=dt)
        big[:, 3:303] = dev(x, dt)
        xt = big[:, 3:303]
        room = torch.full((M, 81), 5.0, device="cuda", dtype=torch.bfloat16)
        y = P.mx4_matmul(xt, wq[:, :160], ws[:, :10], bias=dev(b), y=room[:, 2:77])
        check_product(y, held(f64(xt))[0], wv, b.astype(np.float32), torch.bfloat16)
        assert (room[:, :2] == 5).all() and (room[:, 77:] == 5).all()
        bt, g = dev(b), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = P.mx4_matmul(xt, wq[:, :160], ws[:, :10], bias=bt)
        graphs.append((g, xt, bt, out))
    for i in range(4):
        for g, xt, bt, out in graphs:
            xt.mul_(0.7).add_(0.1)
            bt.mul_(0.9).add_(0.5)
            g.replay()
            want = P.mx4_matmul(xt, wq[:, :160], ws[:, :10], bias=bt)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            check_product(out, held(f64(xt))[0], wv, to_np(bt), xt.dtype)


@pytest.mark.parametrize("M,B", [(1, 37), (6, 37), (40, 37), (90, 37), (300, 37), (6, 13), (40, 16)])
def test_product_any_codes(P, M, B):
    """Rows from elsewhere: every code and scales far apart, also so that sums pass 2^127 in one
    block and 2^-126 in the other direction."""
    say("product codes", M, B)
    g = rng(6, M)
    N = 150
    xq, wq = g.integers(0, 256, (M, 16 * B)), g.integers(0, 256, (N, 16 * B))
    for lo, hi in ((120, 134), (60, 190), (0, 60), (0, 3)):
        xs, ws = g.integers(lo, hi + 1, (M, B)), g.integers(254 - hi, 254 - lo + 1, (N, B))
        if (lo, hi) == (0, 3):
            ws = g.integers(125, 129, (N, B))  # results among the subnormal numbers
        y = P.mx4_matmul(*roomy(xq, xs)[:1], *roomy(wq, ws), x_scale=roomy(xq, xs)[1])
        check_product(y, ref.values(xq, xs), ref.values(wq, ws), None, torch.float32)


@pytest.mark.parametrize("M,K", [(1, 700), (5, 700), (40, 700), (100, 700), (300, 700), (5, 480), (40, 500)])
def test_product_nan_blocks(P, M, K):
    """A NaN scale or number reaches its row (of x) or channel (of w) and nothing else."""
    say("product NaN", M, K)
    x, w, _ = problem(M, K, 90, 1)
    x[M // 2, K - 1], w[17, 3], w[64, K - 50] = np.nan, np.inf, np.nan
    xt = dev(x)
    (xv, _, _), (wv, wc, wE) = held(f64(xt)), held(w)
    assert np.isnan(xv[M // 2]).any() and np.isnan(wv[17]).any()
    y = P.mx4_matmul(xt, *roomy(*ref.pack(wc, wE)))
    check_product(y, xv, wv, None, torch.float32)


def test_product_zero_rows(P):
    say("product zeros")
    x, w, b = problem(9, 320, 50, 2)
    x[3], x[8], w[7] = 0, 0, 0
    wv, wc, wE = held(w)
    y = P.mx4_matmul(dev(x), *roomy(*ref.pack(wc, wE)), bias=dev(b))
    check_product(y, held(f64(dev(x)))[0], wv, b.astype(np.float32), torch.float32)
    assert torch.equal(y[3], dev(b)) and torch.equal(y[8], dev(b))
    empty = P.mx4_matmul(dev(np.zeros((0, 320))), *roomy(*ref.pack(wc, wE)))
    assert empty.shape == (0, 50)


@pytest.mark.parametrize("M", [1, 3, 20, 70, 260])
def test_product_strides_and_rows_between(P, M):
    """Rows of x, w, their scales and y further apart than they are long; what lies between the rows
    of y stays as it was; garbage between the rows of the inputs has no effect."""
    say("product strides", M)
    x, w, b = problem(M, 600, 75, 3)
    wv, wc, wE = held(w)
    pq, pE = ref.pack(wc, wE)
    wq = torch.full((75, 400), 0x77, dtype=torch.uint8, device="cuda")
    ws = torch.full((75, 48), 255, dtype=torch.uint8, device="cuda")
    wq[:, :304], ws[:, :19] = dev(pq, torch.uint8), dev(pE, torch.uint8)
    big = torch.full((M, 777), float("nan"), device="cuda")
    big[:, 3:603] = dev(x)
    room = torch.full((M, 81), 5.0, device="cuda", dtype=torch.bfloat16)
    y = P.mx4_matmul(big[:, 3:603], wq[:, :304], ws[:, :19], bias=dev(b), y=room[:, 2:77])
    assert y.data_ptr() == room[:, 2:77].data_ptr()
    check_product(y, held(f64(big[:, 3:603]))[0], wv, b.astype(np.float32), torch.bfloat16)
    assert (room[:, :2] == 5).all() and (room[:, 77:] == 5).all()
    xq, xs = P.quantize_mx4(dev(x))
    xq2 = torch.full((M, 336), 0x77, dtype=torch.uint8, device="cuda")
    xs2 = torch.full((M, 64), 255, dtype=torch.uint8, device="cuda")
    xq2[:, 16:320], xs2[:, 16:35] = xq, xs
    y2 = P.mx4_matmul(xq2[:, 16:320], wq[:, :304], ws[:, :19], x_scale=xs2[:, 16:35], bias=dev(b),
                      out_dtype=torch.bfloat16)
    assert torch.equal(y2, y)


def test_product_refusals(P):
    say("product refusals")
    x = dev(rng(7).standard_normal((4, 100)))
    wq, ws = P.quantize_mx4(dev(rng(8).standard_normal((20, 100))))
    xq, xs = P.quantize_mx4(x)
    bad = [
        lambda: P.mx4_matmul(x[:, :96], wq, ws), lambda: P.mx4_matmul(x, wq[:, :48], ws),
        lambda: P.mx4_matmul(x, wq, ws.contiguous()), lambda: P.mx4_matmul(x, wq[:, 1:], ws),
        lambda: P.mx4_matmul(x.t(), wq, ws), lambda: P.mx4_matmul(xq, wq, ws),
        lambda: P.mx4_matmul(x, wq, ws, x_scale=xs), lambda: P.mx4_matmul(x, wq, ws, bias=x[0]),
        lambda: P.mx4_matmul(x, wq, ws, out_dtype=torch.int8), lambda: P.mx4_matmul(x, wq.cpu(), ws),
        lambda: P.mx4_matmul(x, wq, ws, y=torch.empty((4, 21), device="cuda")),
        lambda: P.mx4_matmul(xq[:, :48], wq, ws, x_scale=xs[:, :3]),
        lambda: P.mx4_matmul(x.expand(2, 4, 100), wq, ws), lambda: P.mx4_matmul(x, wq, ws, work=x),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    x = dev(rng(7).standard_normal((80, 600)))
    wq, ws = P.quantize_mx4(dev(rng(8).standard_normal((20, 600))))
    with pytest.raises(P.SparseFFNError):
        P.mx4_matmul(x, wq, ws, work=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_product_long_rows(P):
    """Rows of 131071 and more values; offsets of rows of w past 2^32 bytes."""
    say("product long")
    g = rng(9)
    for M, K, N in ((1, 131071, 40), (3, 140000, 20), (70, 70001, 65)):
        x, w, _ = problem(M, K, N, 4, spread=0)
        wv, wc, wE = held(w)
        y = P.mx4_matmul(dev(x), *roomy(*ref.pack(wc, wE)))
        check_product(y, held(f64(dev(x)))[0], wv, None, torch.float32)
    far = 1 << 24  # bytes between rows: row 300 lies behind 2^32
    rows = torch.zeros((300 * far + 4096,), dtype=torch.uint8, device="cuda")
    wq = rows.as_strided((301, 64), (far, 1))
    ws = rows[2048:].as_strided((301, 4), (far, 1))
    x, w, _ = problem(2, 128, 301, 5)
    wv, wc, wE = held(w)
    pq, pE = ref.pack(wc, wE)
    wq.copy_(dev(pq, torch.uint8))
    ws.copy_(dev(pE, torch.uint8))
    for M in (2, 40, 100):
        xt = dev(np.repeat(x, M // 2, axis=0))
        check_product(P.mx4_matmul(xt, wq, ws), held(f64(xt))[0], wv, None, torch.float32)


def test_other_stream_and_graphs(P):
    """A call on another stream; two captured graphs replayed in turn, with eager work between, on
    inputs that change."""
    say("streams, graphs")
    x1, w, b = problem(6, 700, 300, 6)
    x2 = problem(150, 700, 300, 7)[0]
    wq, ws = P.quantize_mx4(dev(w))
    s = torch.cuda.Stream()
    a, c = dev(x1), dev(x2)
    torch.cuda.synchronize()
    e1, e2 = P.mx4_matmul(a, wq, ws), P.mx4_matmul(c, wq, ws)
    y = P.mx4_matmul(a, wq, ws, stream=s)
    q, sc = P.quantize_mx4(c, stream=s)
    z = P.mx4_matmul(q, wq, ws, x_scale=sc, stream=s)
    v = P.dequantize_mx4(q, sc, stream=s)
    s.synchronize()
    assert torch.equal(y, e1) and torch.equal(z, e2)
    assert torch.equal(v, P.dequantize_mx4(*P.quantize_mx4(c)))
    graphs = []
    for t in (a, c):
        g = torch.cuda.CUDAGraph()
        P.mx4_matmul(t, wq, ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = P.mx4_matmul(t, wq, ws)
        graphs.append((g, t, out))
    for i in range(4):
        for g, t, out in graphs:
            t.mul_(0.7).add_(0.1)
            g.replay()
            want = P.mx4_matmul(t, wq, ws)
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_same_bits_every_time(P):
    say("same bits")
    for M, K, N in ((1, 4096, 1000), (12, 4096, 500), (80, 2048, 700), (300, 4096, 1024)):
        x, w, _ = problem(M, K, N, 8)
        wq, ws = P.quantize_mx4(dev(w))
        xt = dev(x, torch.float16)
        first = P.mx4_matmul(xt, wq, ws)
        for _ in range(5):
            assert torch.equal(P.mx4_matmul(xt, wq, ws), first)


@pytest.mark.parametrize("form,rest,M,K,N", mx4_sizes.FORMS)
def test_product_forms(P, form, rest, M, K, N):
    """Each kernel that sizes choose, and products in two launches, on float rows and on rows in blocks,
    against 64-bit products on the device."""
    say("product forms", form, rest, M, K, N)
    gen = torch.Generator("cuda").manual_seed(M + K + N)
    x = torch.randn((M, K), generator=gen, device="cuda").half()
    w = torch.randn((N, K), generator=gen, device="cuda")
    b = torch.randn(N, generator=gen, device="cuda")
    x[M // 2], w[N - 2] = 0, 0
    xq, xs = P.quantize_mx4(x)
    wq, ws = P.quantize_mx4(w)
    xv, wv = P.dequantize_mx4(xq, xs, cols=K).double(), P.dequantize_mx4(wq, ws, cols=K).double()
    room = torch.full((M, N + 3), 9.0, device="cuda")
    y = P.mx4_matmul(x, wq, ws, bias=b, y=room[:, 1:N + 1])
    step = 4096
    for n in range(0, N, step):
        wt = wv[n:n + step].t().contiguous()
        want = torch.matmul(xv, wt) + b[n:n + step].double()
        mag = torch.matmul(xv.abs(), wt.abs()) + b[n:n + step].double().abs()
        lim = (4 * ((K + 127) // 128) + 16) * U * mag + U * want.abs() + 2.0 ** -126
        off = int((~((y[:, n:n + step].double() - want).abs() <= lim)).sum())
        assert off == 0, f"{off} values off from channel {n} on"
    assert (room[:, 0] == 9).all() and (room[:, N + 1:] == 9).all()
    assert torch.equal(P.mx4_matmul(xq, wq, ws, x_scale=xs, bias=b, out_dtype=torch.float32), y)
    assert torch.equal(P.mx4_matmul(x, wq, ws, bias=b, out_dtype=torch.bfloat16), y.to(torch.bfloat16))
    room = torch.full((M, N + 3), 9.0, device="cuda", dtype=torch.float16)
    P.mx4_matmul(xq, wq, ws, x_scale=xs, bias=b, y=room[:, 1:N + 1])
    assert torch.equal(room[:, 1:N + 1], y.half())
    assert (room[:, 0] == 9).all() and (room[:, N + 1:] == 9).all()


def test_many_rows(P):
    """Rows whose codes, values and outputs pass 2^32 bytes, and more of them than a kernel of small tiles
    can be launched for."""
    say("many rows")
    M, K, N = (1 << 26) + 77, 40, 35
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((M, K), generator=gen, device="cuda", dtype=torch.float16)
    w = torch.randn((N, K), generator=gen, device="cuda")
    wq, ws = P.quantize_mx4(w)
    wv = P.dequantize_mx4(wq, ws, cols=K).double().t().contiguous()
    q, s = P.quantize_mx4(x)
    y = P.mx4_matmul(x, wq, ws)
    z = P.mx4_matmul(q, wq, ws, x_scale=s, out_dtype=torch.float16)
    v = P.dequantize_mx4(q, s, cols=K, dtype=torch.float16)
    for r in (0, (1 << 25) - 100, (1 << 26) - 300, M - 513):
        rows = slice(r, r + 513)
        rq, rs = P.quantize_mx4(x[rows].clone())
        assert torch.equal(q[rows], rq) and torch.equal(s[rows], rs)
        rv = P.dequantize_mx4(rq, rs, cols=K)
        assert torch.equal(v[rows], rv.half())
        want = torch.matmul(rv.double(), wv)
        mag = torch.matmul(rv.double().abs(), wv.abs())
        lim = 20 * U * mag + 2.0 ** -11 * want.abs() + 2.0 ** -24
        assert bool(((y[rows].double() - want).abs() <= lim).all())
        assert torch.equal(z[rows], y[rows])
