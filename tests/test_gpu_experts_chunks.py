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


F16, F32 = torch.float16, torch.float32
D = 64


def rows_at(buf, start, pitch, T, dtype):
    """T rows of D values, `pitch` bytes apart from byte `start` of buf on."""
    size = torch.finfo(dtype).bits // 8
    return torch.as_strided(buf.view(dtype), (T, D), (pitch // size, 1), start // size)


@pytest.mark.parametrize("T", [1, 6, 7, 40, 93])
@pytest.mark.parametrize("xs,xp,xt,ys,yp,yt", [
    (0, 256, F32, 0, 256, F32),          # the same rows
    (0, 256, F16, 0, 256, F32),          # rows of the same distance, outputs twice as long
    (0, 256, F32, 0, 128, F16),          # outputs closer together
    (0, 128, F16, 0, 256, F32),          # outputs further apart
    (0, 128, F16, 128, 256, F32),        # and one row ahead
    (0, 256, F32, 256, 256, F32),        # one row ahead
    (512, 256, F32, 0, 256, F32),        # two rows behind
    (0, 512, F32, 256, 512, F32),        # in the gaps between the inputs' rows
    (0, 384, F32, 256, 384, F16),
    (64, 128, F16, 0, 256, F32),
])
def test_outputs_over_inputs_in_chunks(P, T, xs, xp, xt, ys, yp, yt):  # noqa: F811
    say("overlap", T, xs, xp, xt, ys, yp, yt)
    ffn = make_experts(P, 3, D, 96, True, False)
    idx, w = tables(T, 3, 2)
    x = dev(rng(71, T).standard_normal((T, D)), xt)
    want = ffn(x, idx, w, out_dtype=yt)
    for tokens in (7, 1, T):
        buf = torch.zeros(512 + 512 * (T + 2), dtype=torch.uint8, device="cuda")
        over = rows_at(buf, xs, xp, T, xt)
        over.copy_(x)
        y = rows_at(buf, ys, yp, T, yt)
        assert ffn(over, idx, w, y=y, work=ffn.work(tokens, 2)) is y
        assert torch.equal(y, want)


def test_outputs_over_inputs_of_earlier_and_later_chunks(P):  # noqa: F811
    """Outputs further apart that begin before the inputs meet both: refused, unless one chunk
    holds all tokens."""
    T = 40
    say("overlap refused")
    ffn = make_experts(P, 3, D, 96, True, False)
    idx, w = tables(T, 3, 2)
    x = dev(rng(72).standard_normal((T, D)), F16)
    want = ffn(x, idx, w, out_dtype=F32)
    buf = torch.zeros(512 * (T + 2), dtype=torch.uint8, device="cuda")
    over, y = rows_at(buf, 20 * 128, 128, T, F16), rows_at(buf, 0, 256, T, F32)
    over.copy_(x)
    with pytest.raises(P.SparseFFNError):
        ffn(over, idx, w, y=y, work=ffn.work(7, 2))
    assert torch.equal(over, x)
    ffn(over, idx, w, y=y, work=ffn.work(T, 2))
    assert torch.equal(y, want)
