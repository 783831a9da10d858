"""GPU tests of the experts with weight scales of either sign, which callers with 8-bit weights of
their own may bring: relu is taken of the scaled sum. Every kernel form of the activations is
reached. Tolerances as in test_gpu_experts.py."""
import numpy as np
import pytest
import torch

from gpu_util import say
from test_gpu_experts import P, check_experts, dev, make_experts, rng, tables  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,d,f", [(1, 4, 2, 130, 200), (1, 4, 4, 64, 5200), (7, 4, 2, 130, 201), (12, 2, 2, 64, 90),
                                       (150, 3, 1, 200, 170), (400, 2, 2, 130, 333)])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_scales_of_either_sign(P, T, E, k, d, f, gated, bias):  # noqa: F811
    say("signs", T, E, k, d, f, gated, bias)
    ffn = make_experts(P, E, d, f, gated, bias)
    g = rng(60, T, E, d, f)
    for s in (ffn.act_scale, ffn.down_scale):
        s *= dev(g.choice([-1.0, 1.0, 1.0, -0.0], tuple(s.shape)))
    idx, w = tables(T, E, k)
    x = dev(g.standard_normal((T, d)), torch.bfloat16)
    check_experts(P, ffn, x, idx, w, torch.float32)


@pytest.mark.parametrize("T", [1, 9, 90])
def test_gate_scales_that_are_not_finite(P, T):  # noqa: F811
    """relu of minus infinity is 0: only tokens whose gate sum there is not negative become NaN."""
    ffn = make_experts(P, 2, 96, 48, True, False)
    ffn.act_scale[0, 5, 0] = float("inf")
    ffn.act_scale[1, 7, 0] = float("-inf")
    ffn.w_act[1, 7, 0, :] = 0
    ffn.w_act[1, 7, 0, 0] = 100
    idx, w = tables(T, 2, 1, dropped=0.0)
    x = dev(rng(61, T).standard_normal((T, 96)))
    x[:, 0] = 4.0  # the sum of expert 1's row 7 is positive, and its relu 0
    y = check_experts(P, ffn, x, idx, w, torch.float32)
    one = (idx[:, 0] == 1)
    assert bool(torch.isfinite(y[one]).all())


def test_scale_of_a_row_is_a_product(P):  # noqa: F811
    """The scale is the largest magnitude times the 32-bit float nearest to 1 / 127, as the header
    says: not their quotient, which is one last place off for some rows. Largest magnitudes all
    over the range, in the row and by itself."""
    g = rng(62)
    a = (2.0 ** g.uniform(-99, 127, 4000)).astype(np.float32)
    want = (a.astype(np.float64) * float(np.float32(1 / 127))).astype(np.float32)  # 48 bits, rounded once
    quotient = (a.astype(np.float64) / 127).astype(np.float32)
    differ = want != quotient
    assert 40 < int(differ.sum()) < 1000  # about one in twenty
    rows = np.stack([a, -0.75 * a, 0.3 * a], 1)
    for x in (rows, rows[:, ::-1], -rows, a[:, None]):
        q, s = P.quantize_rows(dev(np.ascontiguousarray(x)))
        assert np.array_equal(s.cpu().numpy(), want)
        near = np.rint(x.astype(np.float64) / want[:, None].astype(np.float64))
        assert np.array_equal(q.cpu().numpy(), near)
