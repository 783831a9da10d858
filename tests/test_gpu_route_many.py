"""GPU tests of the router at more tokens than one launch holds: every token is written, and the
choice is the one that 64-bit scores give."""
import pytest
import torch

from gpu_util import say
from test_gpu_experts import P, check_route  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,biased", [((1 << 26) + 7, True), ((1 << 27) + 7, False)])
def test_more_tokens_than_one_launch_holds(P, T, biased):  # noqa: F811
    say("route", T, biased)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    l = torch.empty((T, 2), device="cuda", dtype=torch.float16).normal_(generator=gen)
    bias = torch.tensor([0.25, 0.0], device="cuda") if biased else None
    idx = torch.full((T, 1), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), -9.0, device="cuda")
    P.route(l, 1, score="sigmoid", bias=bias, renormalize=False, idx=idx, weights=w)
    for part in range(0, T, 1 << 24):
        s = l[part:part + (1 << 24)].double()
        s = 1 / (1 + torch.exp(-s))
        c = s if bias is None else s + bias.double()
        want = (c[:, 1] > c[:, 0]).to(torch.int32)
        got = idx[part:part + (1 << 24), 0]
        assert bool((got == want).all()), part
        # |l| is below 8: the exponent's argument and the exponential 10 u, the sum and quotient 2 u
        d = (w[part:part + (1 << 24), 0].double() / s.gather(1, want.long().unsqueeze(1))[:, 0] - 1).abs()
        assert float(d.max()) <= 12 * 2.0 ** -24


@pytest.mark.parametrize("T", [9, 2051])
def test_sigmoids_that_are_zero(P, T):  # noqa: F811
    """Renormalised weights of scores that are zero in 64 bits are zero, however many tokens."""
    say("route zero sigmoids", T)
    rows = torch.tensor([[-800.0, -900.0, -1e30], [-700.0, -709.0, -750.0], [-709.78, -709.783, -710.0],
                         [-100.0, -101.0, -800.0], [0.0, -90.0, -800.0]], device="cuda")
    check_route(P, rows.repeat((T + 4) // 5, 1)[:T].contiguous(), 3, score="sigmoid")


@pytest.mark.parametrize("T", [3, 2049])
@pytest.mark.parametrize("scale", [float("inf"), float("-inf"), float("nan"), 0.0])
@pytest.mark.parametrize("biased", [False, True])
def test_slots_without_an_expert_have_weight_zero(P, T, scale, biased):  # noqa: F811
    """Whatever the weights are multiplied by."""
    say("route empty slots", T, scale, biased)
    l = torch.full((T, 5), -float("inf"), device="cuda")
    l[1:, 2] = 1.0
    for renorm in (True, False):
        idx, w = P.route(l, 3, bias=torch.zeros(5, device="cuda") if biased else None, scale=scale, renormalize=renorm)
        assert bool((idx[0] == -1).all()) and bool((idx[1:] == torch.tensor([2, -1, -1], device="cuda")).all())
        assert bool((w[idx < 0] == 0).all())


@pytest.mark.parametrize("T", [5, 2050])
def test_small_weights_beside_a_small_sum(P, T):  # noqa: F811
    """A score below the normal numbers is a normal one once it is divided by the sum."""
    say("route small weights", T)
    rows = torch.tensor([[-11.5, -89.0, -95.0], [-3.0, -88.9, -89.5], [-13.0, -100.0, -102.0], [-0.5, -89.5, -90.0],
                         [-30.0, -95.0, -110.0]], device="cuda")
    l = rows.repeat(T // 5, 1)
    check_route(P, l, 3, score="sigmoid")
    check_route(P, l, 3, score="sigmoid", bias=torch.tensor([0.5, 0.25, 0.0], device="cuda"))


@pytest.mark.parametrize("T", [4, 2052])
def test_subnormal_logits_are_told_apart(P, T):  # noqa: F811
    """Logits below the normal numbers, and zeros of either sign, which are equal."""
    say("route subnormal", T)
    rows = torch.tensor([[0.0, 1e-40, -1e-40, 3e-45], [-0.0, 0.0, -1e-45, 1e-45], [-1e-42, -2e-42, 0.0, -0.0],
                         [1e-38, 1.1e-38, 1.2e-38, 0.0]], device="cuda")
    check_route(P, rows.repeat(T // 4, 1), 4)
    check_route(P, rows.repeat(T // 4, 1), 3, score="sigmoid", groups=2, top_groups=1)
