"""GPU tests of the router's choice of groups where 32-bit scores cannot decide it: scores that
fp32 holds as subnormal numbers or not at all, and groups whose two scores cancel. The choice is
the 64-bit one (tests/experts_ref.py); weights as in test_gpu_experts.py."""
import numpy as np
import pytest
import torch

from gpu_util import say
from test_gpu_experts import P, check_route, dev, rng  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("score,logits,top_groups", [
    # exact worths of the last two groups 7.43e-44 and 7.52e-44; as fp32 scores 7.6e-44, 7.4e-44
    ("softmax", [[100, 0], [-0.001, -0.001], [0.03, -0.01]], 2),
    # 3.0e-39 and 5.8e-39; as fp32 scores 3.0e-39 and 0, e^88.73 being past the largest fp32 number
    ("sigmoid", [[-88.70, -95], [-88.73, -88.73]], 1),
    ("sigmoid", [[1, 1], [-88.5, -INF], [-88.8, -88.8]], 2),
    # both scores of both groups are below the smallest fp32 number
    ("softmax", [[0, -200], [-130, -130], [-129.5, -INF]], 2),
])
def test_pairs_of_scores_below_the_normal_numbers(P, score, logits, top_groups):  # noqa: F811
    say("pairs", score, logits)
    l = dev(np.array(logits, np.float32).reshape(1, -1))
    G = len(logits)
    for renorm in (True, False):
        check_route(P, l, 2 * G, score=score, groups=G, top_groups=top_groups, group_top=2, renormalize=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups", [(16, 8, 3), (64, 8, 2), (256, 32, 5)])
def test_pairs_of_low_scores(P, score, E, groups, top_groups):  # noqa: F811
    """Worths a few per cent apart where a last place of an fp32 score is as much (a softmax
    whose first group alone is not that far down), or where e^-l passes the largest fp32 number."""
    say("pairs of low scores", score, E, groups)
    T, per = 400, E // groups
    l = (-100 if score == "softmax" else -88.72) + 0.05 * rng(50, E, groups).standard_normal((T, E))
    if score == "softmax":
        l[:, :per] = rng(51, E).uniform(-1, 0, (T, per))
        l[:, 0] = 0
    check_route(P, dev(l), 2 * per, score=score, groups=groups, top_groups=top_groups, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [1.0, 100.0, 1000.0, 3e4])
def test_pairs_whose_biases_cancel(P, score, big):  # noqa: F811
    """A group's two scores carry biases of opposite sign: what fp32 loses in each is many times
    what the groups' worths lie apart."""
    say("cancelling biases", score, big)
    T, E, G = 500, 16, 8
    l = 1e-3 * rng(52, int(big)).standard_normal((T, E))
    bias = dev(np.tile(np.array([big, -big], np.float32), G))
    check_route(P, dev(l), 6, score=score, bias=bias, groups=G, top_groups=3, group_top=2)
    check_route(P, dev(l), 6, score=score, bias=bias, groups=G, top_groups=3, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_pairs_at_the_lowest_value(P, score):  # noqa: F811
    """Biases of the type's lowest value (experts switched off so): a group of two of them is worth
    -6.8e38, which fp32 cannot hold, and still more than a group without any expert."""
    say("lowest biases", score)
    low = float(torch.finfo(torch.float32).min)
    l = dev(np.array([[1, 2, -INF, -INF, 0.5, 1, 1, 2]] * 3, np.float32))
    bias = dev(np.array([0, 0, 0, 0, low, low, low, low], np.float32))
    for group_top in (1, 2):
        for top_groups in (1, 2, 3):
            check_route(P, l, 6, score=score, bias=bias, groups=4, top_groups=top_groups, group_top=group_top)


def test_an_expert_switched_off_by_its_bias_stays_in_the_softmax(P):  # noqa: F811
    """Its score counts in the sum of the others' scores; a logit of minus infinity does not."""
    l = dev(np.array([[1.0, 2.0, 3.0, 0.5], [1.0, 2.0, -INF, 0.5]], np.float32))
    bias = dev(np.array([0, 0, -INF, np.nan], np.float32))
    idx, w = check_route(P, l, 4, bias=bias, renormalize=False)
    assert idx.tolist() == [[1, 0, -1, -1], [1, 0, -1, -1]]
    assert float(w[0].sum()) < 0.4 < 0.8 < float(w[1].sum())
