"""GPU tests of the experts in chunks: more tokens than one chunk may hold, and outputs that lie
over inputs which a later chunk still reads."""
import pytest
import torch

from gpu_util import say
from test_gpu_experts import P, check_experts, dev, make_experts, rng, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def test_more_tokens_than_a_chunk_may_hold(P):  # noqa: F811
    """Scratch for all tokens, of which a chunk takes 2^21: the values of smaller chunks."""
    T = (1 << 21) + 9
    say("experts", T)
    ffn = make_experts(P, 5, 64, 48, True, False)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(70)
    x = torch.empty((T, 64), device="cuda", dtype=torch.float16).normal_(generator=gen)
    idx = torch.randint(-1, 6, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.rand((T, 1), generator=gen, device="cuda")
    y = ffn(x, idx, w, work=ffn.work(T, 1))
    assert torch.equal(y, ffn(x, idx, w))
    pick = [0, 1, 1 << 20, (1 << 21) - 1, 1 << 21, T - 1]
    check_experts(P, ffn, x[pick], idx[pick], w[pick], torch.float16, y=y[pick])
