"""GPU tests of rows in 4-bit blocks and their products at the greatest length, 2^20, and just below it.

A bound on the roundings of so many sums would say little, so the numbers are such that there are none: codes
for 0, 0.5, 1, 1.5 and 2 and scales of 1 and 1/2 have products that are multiples of 1/16, and while the
magnitudes of a row's products add up to less than 2^24 / 16 every partial sum is one of these multiples and
held exactly in 32 bits, in any order. Outputs have to be equal."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from gpu_util import say, to_np

pytestmark = pytest.mark.gpu
LONGEST = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def P():
    import activation_sparse_decode_rank_amd as P  # fails loudly without the HIP library
    torch.cuda.init()
    yield P


def held(rows, gen):
    """Codes and scales of rows of the greatest length."""
    half = lambda: (torch.randint(0, 5, (rows, LONGEST // 2), generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
                    + 8 * torch.randint(0, 2, (rows, LONGEST // 2), generator=gen, device="cuda", dtype=torch.uint8))
    return half() + 16 * half(), torch.randint(126, 128, (rows, LONGEST // 32), generator=gen, device="cuda",
                                               dtype=torch.uint8)


def values(q, s):
    """Their values, from the codes themselves: half the code, times the scale."""
    c = torch.stack((q & 15, q >> 4), 2).reshape(q.shape[0], -1)
    v = torch.where(c >= 8, 8.0 - c.double(), c.double()) / 2
    return (v.view(q.shape[0], -1, 32) * torch.exp2(s.double() - 127).unsqueeze(2)).view(q.shape[0], -1)


# few rows, some, tens and hundreds; channels for the tiles that share their length among waves and for those
# that do not
@pytest.mark.parametrize("M,N", [(1, 1), (1, 17), (4, 333), (1, 8599), (33, 8599), (67, 2003), (130, 12001),
                                 (842, 12001)])
@pytest.mark.parametrize("K", [LONGEST, LONGEST - 5])
def test_products(P, M, N, K):
    say("longest products", M, N, K)
    gen = torch.Generator("cuda").manual_seed(M + N)
    xq, xs = held(M, gen)
    wq, ws = held(N, gen)
    x = values(xq, xs)
    if K < LONGEST:
        x[:, K:] = 0
    b = torch.randint(-64, 65, (N,), generator=gen, device="cuda").float() / 16
    want, most = torch.empty((M, N), dtype=torch.float64, device="cuda"), 0.0
    for n in range(0, N, 512):
        w = values(wq[n:n + 512], ws[n:n + 512])
        want[:, n:n + 512] = torch.matmul(x, w.t().contiguous()) + b[n:n + 512].double()
        if n == 0:
            most = float(torch.matmul(x.abs(), w.abs().t().contiguous()).max()) + 4
    assert most < 0.95 * 2 ** 20  # of the first channels; the others' lie within a few thousandths of these
    xt = x[:, :K].bfloat16()
    assert torch.equal(xt.double(), x[:, :K])
    y = P.mx4_matmul(xt, wq, ws, bias=b, out_dtype=torch.float32)
    assert torch.equal(y.double(), want)
    if K == LONGEST:
        assert torch.equal(P.mx4_matmul(xq, wq, ws, x_scale=xs, bias=b), y)
        assert torch.equal(P.mx4_matmul(xq, wq, ws, x_scale=xs, bias=b, out_dtype=torch.bfloat16), y.bfloat16())


@pytest.mark.parametrize("K", [LONGEST, LONGEST - 5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_blocks(P, K, dtype):
    say("longest blocks", K, dtype)
    x = torch.randn((2, K), device="cuda", generator=torch.Generator("cuda").manual_seed(K)).to(dtype)
    q, s = P.quantize_mx4(x)
    rq, rs = ref.pack(*ref.blocks(x.cpu().double().numpy()))
    assert np.array_equal(to_np(q), rq) and np.array_equal(to_np(s), rs)
    want = torch.from_numpy(ref.values(rq, rs)[:, :K])
    assert torch.equal(P.dequantize_mx4(q, s, cols=K).double().cpu(), want)
    assert torch.equal(P.dequantize_mx4(q, s, cols=K, dtype=dtype).cpu(), want.to(dtype))


def test_longer_ones_are_refused(P):
    say("longer")
    x = torch.zeros((1, LONGEST + 32), device="cuda")
    q, s = P.quantize_mx4(x)  # rows may be longer than a product takes
    for call in (lambda: P.mx4_matmul(x, q, s), lambda: P.mx4_matmul(q, q, s, x_scale=s)):
        with pytest.raises(P.SparseFFNError):
            call()
