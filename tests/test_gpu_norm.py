"""GPU tests of the norm in front of 8- and 4-bit products (rms_norm) against its plain 64-bit form
(tests/mx4_ref.py), against the library's own quantisers, and in a run of the operators together.

Tolerances, each from the roundings made:
 - v = x + residual rounded to x's type: equal to torch's sum, whose one rounding is the same;
 - float outputs: 64-bit arithmetic, whose errors (some 2^-50) are far below half a step of the
   output type, then one rounding: half a step of the value (of the smallest normal below that),
   times 1 + 2^-20 for where the 64-bit value lies next to the middle of two steps;
 - 8-bit rows and 4-bit blocks: equal to what quantize_rows and quantize_mx4 give for the fp32
   output of the same call."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from gpu_util import say, to_np

pytestmark = pytest.mark.gpu
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


def check(got, want, dtype):
    got = f64(got)
    fi = torch.finfo(dtype)
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(got), bad)
    over = np.abs(want) >= fi.max * (1 + fi.eps / 4)
    with np.errstate(invalid="ignore"):
        d = np.abs(got - want)[~bad & ~over]
    lim = (fi.eps / 2 * (1 + 2.0 ** -20) * np.maximum(np.abs(want), fi.tiny))[~bad & ~over]
    off = int((~(d <= lim)).sum())
    assert off == 0, f"{off} values off, worst {np.max(d / lim):.3g} of the bound"
    assert np.isinf(got[over]).all()


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float(), -7.0), torch.nan_to_num(b.float(), -7.0))


def check_norm(P, x, w, res, eps=1e-6):
    """Every output form of one call's inputs."""
    kw = dict(eps=eps)
    if res is not None:
        kw["residual"] = res
    v = x if res is None else x + res
    want = ref.norm(f64(v), None if w is None else f64(w), eps)
    for out in DT.values():
        got = P.rms_norm(x, w, out=out, **kw)
        if res is not None:
            got, s = got
            assert s.dtype == x.dtype and same(s, v)
        assert got.dtype == out and got.shape == x.shape
        check(got, want, out)
    y = P.rms_norm(x, w, out=torch.float32, **kw)
    y = y if res is None else y[0]
    q, s, *r = P.rms_norm(x, w, out="i8", **kw)
    q2, s2 = P.quantize_rows(y)
    assert same(s, s2) and torch.equal(q, q2) and q.stride() == q2.stride()
    assert res is None or same(r[0], v)
    q, s, *r = P.rms_norm(x, w, out="mx4", **kw)
    q2, s2 = P.quantize_mx4(y)
    assert torch.equal(s, s2) and torch.equal(q, q2) and s.stride() == s2.stride()
    assert res is None or same(r[0], v)


@pytest.mark.parametrize("d", [1, 2, 7, 8, 17, 31, 32, 33, 64, 100, 511, 768, 1000, 1013, 1024, 1025,
                               2048, 4096, 4097, 5120, 11008, 12288, 16384, 16385, 40000])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_sizes(P, d, dtype):
    say("norm", d, dtype)
    for T in (1, 2, 37 if d < 20000 else 3):
        g = rng(1, d, T)
        x = dev(g.standard_normal((T, d)) * 2.0 ** g.integers(-6, 7, (T, 1)), DT[dtype])
        res = dev(g.standard_normal((T, d)) * 3, DT[dtype])
        w = dev(1 + 0.3 * g.standard_normal(d), DT[dtype])
        check_norm(P, x, w, res)
        check_norm(P, x, None if T == 2 else w.float(), None, eps=1e-3)
        check_norm(P, x, w.half() if T == 1 else w.bfloat16(), res, eps=0.0)


@pytest.mark.parametrize("d", [96, 3000, 9000, 20000])
def test_far_values(P, d):
    """Rows of zeros, subnormal and largest numbers, infinities and NaN, beside ordinary rows;
    weights of zero and of either sign."""
    say("norm far", d)
    g = rng(2, d)
    x = g.standard_normal((12, d)).astype(np.float32)
    x[0] = 0
    x[1] = 2.0 ** -149
    x[2] = g.standard_normal(d) * 2.0 ** -110
    x[3] = g.choice([-1, 1], d) * np.finfo(np.float32).max
    x[4] = g.standard_normal(d) * 2.0 ** 100
    x[5, d // 2] = np.inf
    x[6, d - 1] = np.nan
    x[7, 0] = 1e30
    x[8] *= 1e-25
    w = g.standard_normal(d)
    w[3], w[d - 2] = 0, -5
    for eps in (1e-6, 0.0, 1e-30):
        check_norm(P, dev(x), dev(w), None, eps)
    check_norm(P, dev(x), None, dev(np.roll(x, 1, axis=0)))
    for bad in (np.inf, -np.inf, np.nan, 1e38):  # reaches that column, and every number held with it
        wb = w.copy()
        wb[d // 3] = bad
        check_norm(P, dev(x), dev(wb), None)
    h = x[[0, 2, 5, 6, 9, 10, 11]] * np.float32(3)
    for dt in ("f16", "bf16"):
        check_norm(P, dev(h, DT[dt]), dev(w, DT[dt]), dev(h[::-1] * 100, DT[dt]))


def test_sum_is_rounded_once_and_before_the_norm(P):
    """bf16 sums that lie between two steps, and a residual so large that x alone is lost."""
    say("norm sums")
    g = rng(3)
    x = dev(g.standard_normal((64, 512)), torch.bfloat16)
    res = dev(g.choice([-1.0, 1.0], (64, 512)) * 256 + g.integers(-3, 4, (64, 512)) * 0.5, torch.bfloat16)
    check_norm(P, x, None, res)


def test_strides_and_shapes(P):
    say("norm strides")
    g = rng(4)
    big = dev(g.standard_normal((9, 500)), torch.float16)
    other = dev(g.standard_normal((9, 400)), torch.float16)
    check_norm(P, big[:, 3:203], dev(g.standard_normal(200)), other[:, 7:207])
    check_norm(P, big[::2, :77], None, other[::2, :77])
    check_norm(P, big[2:3, :77], None, None)
    x = dev(g.standard_normal((2, 3, 70)))
    r = dev(g.standard_normal((2, 3, 70)))
    y, v = P.rms_norm(x, residual=r)
    y2, v2 = P.rms_norm(x.view(6, 70), residual=r.view(6, 70))
    assert y.shape == x.shape and torch.equal(y.view(6, 70), y2) and torch.equal(v.view(6, 70), v2)
    q, s = P.rms_norm(x, out="i8")
    assert q.shape == x.shape and s.shape == (2, 3)
    q, s = P.rms_norm(x, out="mx4")
    assert q.shape == (2, 3, 48) and s.shape == (2, 3, 3)
    assert torch.equal(P.rms_norm(x.transpose(0, 1)), P.rms_norm(x).transpose(0, 1))
    assert torch.equal(P.rms_norm(x[0, 0]), P.rms_norm(x)[0, 0])
    assert P.rms_norm(x[:, :0]).shape == (2, 0, 70)


@pytest.mark.parametrize("d", [70, 2500, 7000, 20001])
def test_in_place_sums(P, d):
    """The sum over the residual and over x, and between rows that stay as they were."""
    say("norm in place", d)
    g = rng(5, d)
    x, r = dev(g.standard_normal((5, d)), torch.bfloat16), dev(g.standard_normal((5, d)), torch.bfloat16)
    for out in (torch.bfloat16, "i8", "mx4"):
        want = P.rms_norm(x, residual=r, out=out)
        r2, x2 = r.clone(), x.clone()
        got = P.rms_norm(x, residual=r2, out=out, residual_out=r2)
        assert got[-1].data_ptr() == r2.data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = P.rms_norm(x2, residual=r, out=out, residual_out=x2)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        room = torch.full((5, d + 9), 2.0, dtype=torch.bfloat16, device="cuda")
        got = P.rms_norm(x, residual=r, out=out, residual_out=room[:, 4:d + 4])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (room[:, :4] == 2).all() and (room[:, d + 4:] == 2).all()


def test_rows_between_outputs(P):
    """Bytes behind the rows of every output form, through the C call."""
    say("norm between rows")
    N = P._native
    x = dev(rng(6).standard_normal((4, 70)))
    for kind, ld, esz, end in ((N.SFFN_F32, 75, 4, 70), (N.SFFN_F16, 75, 2, 70), (N.SFFN_I8, 112, 1, 80),
                               (N.SFFN_MX4, 64, 1, 48)):
        y = torch.full((4, ld * esz), 0x55, dtype=torch.uint8, device="cuda")
        s = torch.full((4, 16), 0x55, dtype=torch.uint8, device="cuda")
        sc = s.data_ptr() if kind >= N.SFFN_I8 else None
        N.sparse_ffn_rms_norm(x.data_ptr(), 0, 70, None, 0, 4, 70, None, 0, 1e-6, None, 0, y.data_ptr(), kind,
                              ld, sc, 16, 0)
        torch.cuda.synchronize()
        assert (y[:, end * esz:] == 0x55).all()
        if kind == N.SFFN_I8:
            assert (y[:, 70:80] == 0).all() and (s.view(-1)[16:] == 0x55).all()
        if kind == N.SFFN_MX4:
            assert (s[:, 3:] == 0x55).all()


@pytest.mark.parametrize("d", [70, 3000, 20001])
def test_outputs_over_inputs(P, d):
    """Through the C call: a float y of x's type over x or over the residual, with the sum elsewhere or
    over the other one."""
    say("norm over inputs", d)
    N = P._native
    g = rng(11, d)
    x0, r0 = dev(g.standard_normal((9, d)), torch.bfloat16), dev(g.standard_normal((9, d)), torch.bfloat16)
    plain = P.rms_norm(x0)
    y0, v0 = P.rms_norm(x0, residual=r0)

    def call(x, r, v, y):
        N.sparse_ffn_rms_norm(x.data_ptr(), N.SFFN_BF16, d, None if r is None else r.data_ptr(), d, 9, d, None, 0,
                              1e-6, None if v is None else v.data_ptr(), d, y.data_ptr(), N.SFFN_BF16, d, None, 0, 0)
        torch.cuda.synchronize()

    x = x0.clone()
    call(x, None, None, x)
    assert torch.equal(x, plain)
    x, r, v = x0.clone(), r0.clone(), torch.empty_like(x0)
    call(x, r, v, x)
    assert torch.equal(x, y0) and torch.equal(v, v0) and torch.equal(r, r0)
    x, r, v = x0.clone(), r0.clone(), torch.empty_like(x0)
    call(x, r, v, r)
    assert torch.equal(r, y0) and torch.equal(v, v0) and torch.equal(x, x0)
    x, r = x0.clone(), r0.clone()
    call(x, r, r, x)
    assert torch.equal(x, y0) and torch.equal(r, v0)
    x, r = x0.clone(), r0.clone()
    call(x, r, x, r)
    assert torch.equal(r, y0) and torch.equal(x, v0)


def test_refusals(P):
    say("norm refusals")
    x = dev(rng(7).standard_normal((4, 64)))
    for call in (lambda: P.rms_norm(x, x[0, :60]), lambda: P.rms_norm(x, x[0].long()),
                 lambda: P.rms_norm(x, x[0].cpu()), lambda: P.rms_norm(x, residual=x.half()),
                 lambda: P.rms_norm(x, residual=x[:3]), lambda: P.rms_norm(x, residual=x.cpu()),
                 lambda: P.rms_norm(x, residual=x, residual_out=x[:3]),
                 lambda: P.rms_norm(x, residual=x, residual_out=x.t().contiguous().t()),
                 lambda: P.rms_norm(x, out=torch.int8), lambda: P.rms_norm(x, out="fp4"),
                 lambda: P.rms_norm(x[:, :0])):
        with pytest.raises(ValueError):
            call()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(P.SparseFFNError):
            P.rms_norm(x, eps=eps)


def test_many_rows(P):
    """More rows than workgroups in one launch."""
    say("norm many rows")
    T = (1 << 20) + 77
    x = torch.randn((T, 8), device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(1))
    y = P.rms_norm(x, out=torch.float32)
    v = x.double()
    want = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    assert ((y.double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -20) * want.abs()).all()
    q, s = P.quantize_mx4(y)
    q2, s2 = P.rms_norm(x, out="mx4")
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_streams_and_graphs(P):
    say("norm streams")
    g = rng(8)
    x, r, w = dev(g.standard_normal((50, 3000)), torch.float16), dev(g.standard_normal((50, 3000)),
                                                                  torch.float16), dev(g.standard_normal(3000))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = P.rms_norm(x, w, residual=r, out="i8")
    got = P.rms_norm(x, w, residual=r, out="i8", stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for out in ("i8", "mx4", torch.float16):
        h = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(h):
            held = P.rms_norm(x, w, residual=r, out=out)
        graphs.append((h, out, held))
    for _ in range(3):
        x.mul_(0.9).add_(0.01)
        for h, out, held in graphs:
            h.replay()
            want = P.rms_norm(x, w, residual=r, out=out)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("T", [1, 3, 24, 130])
@pytest.mark.parametrize("bits", ["i8", "mx4"])
def test_a_layer_of_them(P, T, bits):
    """Norm, up and gate products, ReLU, down product, and the next norm with its residual, as a
    decoder's layer runs them, against the same mathematics in 64 bits on the values held. The
    products' outputs decide 8- and 4-bit numbers further on, so each step is checked from the
    inputs that it was given."""
    say("layer", T, bits)
    g = rng(9, T)
    d, f = 512, 1376
    x = dev(g.standard_normal((T, d)), torch.bfloat16)
    res = dev(g.standard_normal((T, d)) * 2, torch.bfloat16)
    n1 = dev(1 + 0.1 * g.standard_normal(d), torch.bfloat16)
    hold = P.quantize_rows if bits == "i8" else P.quantize_mx4
    product = P.i8_matmul if bits == "i8" else P.mx4_matmul
    weights = [hold(dev(g.standard_normal(s) * 0.05)) for s in ((f, d), (f, d), (d, f))]

    def values(q, s):
        return f64(q) * f64(s)[:, None] if bits == "i8" else ref.values(to_np(q), to_np(s))

    def checked(got, q, s, w, dtype):
        a, b = values(q, s), values(*w)
        n = min(a.shape[1], b.shape[1])
        want, mag = ref.matmul(a[:, :n], b[:, :n])
        err = (4 * ((n + 127) // 128) + 16) * 2.0 ** -24 * mag
        lim = err + torch.finfo(dtype).eps / 2 * (np.abs(want) + err) + 1e-30
        assert (np.abs(f64(got) - want) <= lim).all()

    q, s, r = P.rms_norm(x, n1, residual=res, out=bits)
    assert torch.equal(r, x + res)
    gate = product(q, *weights[0], x_scale=s, out_dtype=torch.float32)
    up = product(q, *weights[1], x_scale=s, out_dtype=torch.float32)
    checked(gate, q, s, weights[0], torch.float32)
    checked(up, q, s, weights[1], torch.float32)
    h = torch.relu(gate) * up
    y = product(h, *weights[2], out_dtype=torch.bfloat16)
    hq, hs = hold(h)
    checked(y, hq, hs, weights[2], torch.bfloat16)
    assert torch.equal(y, product(hq, *weights[2], x_scale=hs, out_dtype=torch.bfloat16))
    out, r2 = P.rms_norm(y, n1, residual=r, residual_out=r)
    assert r2.data_ptr() == r.data_ptr() and torch.equal(r2, y + (x + res))
    check(out, ref.norm(f64(r2), f64(n1)), torch.bfloat16)


@pytest.mark.parametrize("shape", [(1, 40), (5, 64), (3, 4, 100), (77,), (0, 33), (2, 0, 33), (6, 1)])
def test_both_ways_to_the_library(P, shape, monkeypatch):
    """The extension module's calls and the functions' own give the same bits, shapes and strides; a
    regular call takes the first way."""
    import sys
    say("both ways", shape)
    M = sys.modules["activation_sparse_decode_rank_amd.mx4"]
    g = rng(10, *shape)
    x, r = dev(g.standard_normal(shape), torch.float16), dev(g.standard_normal(shape), torch.float16)
    w = dev(g.standard_normal(shape[-1]))
    n = int(np.prod(shape[:-1], dtype=np.int64))

    class Off:
        def __getattr__(self, name):
            return lambda *a: None

    def calls():
        out = []
        for kind in (None, torch.float32, "i8", "mx4"):
            for res in (None, r):
                got = P.rms_norm(x, w, residual=res, out=kind)
                out += list(got) if isinstance(got, tuple) else [got]
        out += list(P.rms_norm(x, residual=r, residual_out=torch.empty_like(x)))
        q, s = P.quantize_mx4(x)
        out += [q, s, P.dequantize_mx4(q, s, cols=shape[-1]), P.dequantize_mx4(q, s, dtype=torch.bfloat16)]
        if n:
            x2 = x.reshape(n, shape[-1])
            q2, s2 = P.quantize_mx4(x2)
            b = dev(np.arange(n))
            out += [P.mx4_matmul(x2, q2, s2), P.mx4_matmul(q2, q2, s2, x_scale=s2, bias=b),
                    P.mx4_matmul(x2, q2, s2, out_dtype=torch.bfloat16)]
        return out

    fast = calls()
    monkeypatch.setattr(M, "_calls", Off())
    slow = calls()
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b)
        assert a.numel() == 0 or a.stride() == b.stride()
    monkeypatch.undo()
    if n and len(shape) == 2:
        def no(*a):
            raise AssertionError("the ctypes way was taken")
        for f in ("sparse_ffn_rms_norm", "sparse_ffn_quantize_mx4", "sparse_ffn_dequantize_mx4",
                  "sparse_ffn_mx4_matmul"):
            monkeypatch.setattr(M.N, f, no)
        calls()
