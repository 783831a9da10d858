"""GPU tests of the norm's float outputs by their bits: y = v w / sqrt(mean(v^2) + eps) in 64 bits, rounded
once to the output's type.

The kernel's and the reference's 64-bit values differ: their sums add at most 40 + 6 + 16 (a thread's values,
a wave's lanes, the waves of a workgroup) and some 30 (numpy's) numbers one behind the other, which the root
halves, and a few more roundings follow: together less than 100 of them, 100 * 2^-53 < 2^-46 of the value.
So either neighbour will do within 2^-45 of the middle of two, and nowhere else."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import norm_round as nr
from gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def P():
    import activation_sparse_decode_rank_amd as P  # fails loudly without the HIP library
    torch.cuda.init()
    yield P


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("d", [8, 64, 1000, 1024, 4096, 8192, 16384, 20000])
@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_beside_the_middle_of_two_outputs(P, d, out):
    """Rows whose mean square is 1 exactly (of 8 values three are 1.5, five 0.5) and eps 0: y = v w, with
    weights that bring 1.5 w beside the middles of neighbouring outputs."""
    say("rounding middles", d, out)
    g = np.random.Generator(np.random.PCG64([1, d]))
    w = nr.beside_middles(out, g, max(d // 3 + 1, 8))[0]
    w = g.permutation(w)[:d]
    x = np.stack([np.roll(np.tile([1.5, 1.5, 1.5, .5, .5, .5, .5, .5], d // 8), r) for r in range(8)])
    x *= g.choice([-1.0, 1.0], x.shape)
    y = x * w.astype(np.float64)
    if d >= 64:
        with np.errstate(over="ignore"):
            assert nr.off(nr.once(y.astype(np.float32).astype(np.float64), out), y, out) >= d // 32
    for kind, dt in DT.items():
        xt = dev(x, dt)
        got = P.rms_norm(xt, dev(w), eps=0.0, out=DT[out])
        assert nr.off(f64(got), y, out) == 0, kind
        half, zero = dev(x / 2, dt), torch.zeros_like(xt)
        got, s = P.rms_norm(half, dev(w), residual=half, eps=0.0, out=DT[out])
        assert torch.equal(s, xt) and nr.off(f64(got), y, out) == 0, kind
        y3 = P.rms_norm(xt, dev(w), residual=zero, eps=0.0, out=torch.float32)[0]
        assert nr.off(f64(y3), y, "f32") == 0, kind


@pytest.mark.parametrize("T,d", [(7, 33), (300, 1013), (256, 4096), (21, 12288), (9, 16385), (5, 40000)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_every_output_is_rounded_once(P, T, d, dtype):
    say("rounding", T, d, dtype)
    g = np.random.Generator(np.random.PCG64([2, T, d]))
    x, r = dev(g.standard_normal((T, d)), DT[dtype]), dev(3 * g.standard_normal((T, d)), DT[dtype])
    for w in (dev(1 + 0.2 * g.standard_normal(d)), dev(1 + 0.2 * g.standard_normal(d), DT[dtype]), None):
        for res in (None, r):
            v = x if res is None else x + res
            want = ref.norm(f64(v), None if w is None else f64(w), 1e-6)
            for out, dt in DT.items():
                got = P.rms_norm(x, w, residual=res, out=dt)
                assert nr.off(f64(got if res is None else got[0]), want, out) == 0, out


def test_outputs_out_of_range(P):
    """Outputs above fp16's largest number and below its normal ones, infinities and NaN, by their bits."""
    say("rounding far")
    g = np.random.Generator(np.random.PCG64(3))
    x = g.standard_normal((64, 520)).astype(np.float32)
    w = (g.standard_normal(520) * 2.0 ** g.integers(-40, 18, 520)).astype(np.float32)
    far = (g.standard_normal(520) * 2.0 ** g.integers(-148, 126, 520)).astype(np.float32)
    x[3, 5], x[9, 0], x[11] = np.inf, np.nan, 0
    for weights, out in ((w, "f16"), (far, "bf16"), (far, "f32")):
        want = ref.norm(x.astype(np.float64), weights.astype(np.float64), 1e-6)
        got = P.rms_norm(dev(x), dev(weights), out=DT[out])
        assert nr.off(f64(got), want, out) == 0, out
