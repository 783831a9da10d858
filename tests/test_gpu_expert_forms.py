"""GPU tests of every kernel form that the expert-layer operators choose from by size: the router
with two tokens a wave, products of few rows with a wave for each tile, and each tile of many rows
in the plain, gated and down products. Whole outputs against 64-bit forms in elementary torch
operations; tolerances as in test_gpu_experts.py."""
import pytest
import torch

import experts_ref as ref
from gpu_util import say, to_np
from test_gpu_experts import DT, P, U, check, check_route, dev, f64, logits_of, make_experts, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def held(x):
    """Rows in 8 bits: whole numbers and scales in 64 bits (see the header for the definition)."""
    x = x.double()
    a = x.abs().amax(1)
    s = (a.float() * torch.tensor(1 / 127, dtype=torch.float32)).double()
    s = torch.where(a < 2.0 ** -100, 0.0, s)
    return torch.where(s.unsqueeze(1) > 0, torch.round(x / s.unsqueeze(1)), 0.0), s


def matmul_of(q, s, w, ws, bias=None):
    p = (q @ w.double().t().contiguous()) * s.unsqueeze(1) * ws.double()
    b = torch.zeros_like(ws.double()) if bias is None else bias.double()
    return p + b, p.abs() + b.abs()


def experts_of(ffn, x, idx, weights):
    T, d = x.shape
    q, s = held(x)
    y, mag = torch.zeros((T, d), dtype=torch.float64, device="cuda"), torch.zeros((T, d), dtype=torch.float64, device="cuda")
    for e in range(ffn.n_experts):
        t, slot = torch.nonzero(idx == e, as_tuple=True)
        if not t.numel():
            continue
        wa = ffn.w_act[e].double().reshape(-1, d)
        a = (q[t] @ wa.t().contiguous()) * (s[t].unsqueeze(1) * ffn.act_scale[e].double().reshape(-1))
        if ffn.gated:
            g, u = a[:, ::2], a[:, 1::2]
        else:
            g, u = a, 1.0
        if ffn.b_act is not None:
            g = g + ffn.b_act[e].double()
        h = (torch.clamp_min(g, 0.0) * u).float().double()
        hq, hs = held(h)
        p = (hq @ ffn.w_down[e].double().t().contiguous()) * hs.unsqueeze(1) * ffn.down_scale[e].double()
        p = p * weights[t, slot].double().unsqueeze(1)
        y.index_put_((t,), p, accumulate=True)
        mag.index_put_((t,), p.abs(), accumulate=True)
    return y.cpu().numpy(), mag.cpu().numpy()


def experts_in_a_window(P, ffn, T, E, k, d, xt, yt, dropped, seed):  # noqa: F811
    """The call on random tables, in one chunk, its output a window of a larger tensor at an odd
    column."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    idx = torch.randint(0, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    idx[torch.rand((T, k), generator=gen, device="cuda") < dropped] = -1
    w = torch.rand((T, k), generator=gen, device="cuda")
    x = torch.randn((T, d), generator=gen, device="cuda").to(DT[xt])
    out = torch.full((T + 2, d + 9), -7.0, dtype=DT[yt], device="cuda")
    ffn(x, idx, w, y=out[1:-1, 3:3 + d], work=ffn.work(T, k))
    want, mag = experts_of(ffn, x, idx, w)
    check(out[1:-1, 3:3 + d], want, (k + 4) * U * mag, DT[yt])
    out[1:-1, 3:3 + d] = -7.0
    assert (out == -7.0).all()


@pytest.mark.parametrize("T,E,k,d,f", [
    (1, 10, 8, 300, 2600), (1, 20, 16, 300, 2600),   # one token, a wave for each tile of its slots
    (16, 64, 8, 600, 610), (40, 64, 8, 600, 610),    # a decode batch over many small experts
    (768, 64, 1, 410, 390), (1792, 64, 1, 410, 390),  # up to 16 and 32 rows, a wave a tile
    (20, 3, 2, 4500, 100), (20, 3, 2, 17000, 100),   # long rows into 8 bits, and longer than a workgroup holds
    (1920, 64, 2, 600, 600),                         # 64 rows x 128 channels
    (56320, 512, 1, 600, 300),                       # 128 x 256
    (102400, 512, 1, 600, 300),                      # 256 x 256
])
@pytest.mark.parametrize("gated", [True, False])
def test_experts_in_every_form(P, T, E, k, d, f, gated):  # noqa: F811
    say("forms", T, E, k, d, f, gated)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(80)
    rand = lambda *n: torch.randn(n, generator=gen, device="cuda") * 0.05  # noqa: E731
    ffn = P.ExpertFFN.from_float(w_act=rand(E, f, d), w_up=rand(E, f, d) if gated else None, w_down=rand(E, d, f),
                                 b_act=None if gated else rand(E, f) * 6)
    for xt, yt in (("f32", "f32"), ("bf16", "f16")):
        experts_in_a_window(P, ffn, T, E, k, d, xt, yt, 0.05, T + k)


@pytest.mark.parametrize("M,K,N", [(1, 300, 41003), (4, 300, 41003), (5, 129, 41003), (16, 513, 41003), (17, 513, 41003),
                                   (32, 300, 41003), (8, 256, 128256), (3, 8208, 41003), (9, 8208, 41003), (30, 8208, 41003)])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("f16", "bf16"), ("i8", "f16")])
def test_matmul_of_many_channels(P, M, K, N, xt, yt):  # noqa: F811
    """As many channels as a vocabulary, few rows: a wave for each tile up to 8192 values."""
    say("many channels", M, K, N, xt, yt)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M * K)
    w, ws = P.quantize_rows(torch.randn((N, K), generator=gen, device="cuda") * 0.02)
    b = torch.randn(N, generator=gen, device="cuda")
    x = torch.randn((M, K), generator=gen, device="cuda").to(DT.get(xt, torch.float32))
    xs = None
    if xt == "i8":
        x, xs = P.quantize_rows(x)
    out = torch.full((M + 2, N + 9), -7.0, dtype=DT[yt], device="cuda")
    P.i8_matmul(x, w, ws, x_scale=xs, bias=b, y=out[1:-1, 3:3 + N])
    q, s = held(x) if xs is None else (x.double(), xs.double())
    want, mag = matmul_of(q, s, w, ws, b)
    check(out[1:-1, 3:3 + N], want.cpu().numpy(), 4 * U * mag.cpu().numpy(), DT[yt])
    out[1:-1, 3:3 + N] = -7.0
    assert (out == -7.0).all()


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (33, 4), (64, 8), (65, 32), (128, 3), (129, 6), (160, 6), (161, 5), (256, 8)])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "far"])
def test_route_of_many_tokens(P, E, k, kind):  # noqa: F811
    """From 2048 tokens on the plain choice goes two tokens a wave: an odd number of them, also in
    the last workgroup."""
    say("route many", E, k, kind)
    for i, score in enumerate(("softmax", "sigmoid")):
        dt = ("f32", "f16", "bf16")[(E + i) % 3]
        l = logits_of(2049 + 4 * i, E, dt, k, kind)
        check_route(P, l, k, score=score, renormalize=(E + i) % 2 == 0, scale=2.5 if i else 1.0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k", [(30011, 160, 6), (2048, 256, 32), (9001, 64, 8)])
def test_route_ties_of_many_tokens(P, T, E, k, dtype):  # noqa: F811
    """Logits of few different values: ties go to the lowest index, in every token."""
    say("route many ties", T, E, k, dtype)
    l = dev(rng(81, T, E).integers(-3, 4, (T, E)).astype("float32"), DT[dtype])
    l[::5, ::3] = -float("inf")
    l[7] = -float("inf")
    idx, w = P.route(l, k, renormalize=False)
    c, want = torch.sort(l.double(), dim=1, descending=True, stable=True)
    want = torch.where(c > -float("inf"), want, -1)[:, :k]
    assert bool((idx == want).all())
    s = torch.where(c > -float("inf"), torch.exp(c - c[:, :1]), 0.0)
    s = torch.nan_to_num(s / s.sum(1, keepdim=True))[:, :k]
    assert bool(((w.double() - s).abs() <= (2 * 6 + 100) * U * s).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "far"])
def test_route_of_many_tokens_with_groups(P, score, kind):  # noqa: F811
    say("route many groups", score, kind)
    T, E = 2051, 64
    b = dev(rng(82).integers(-1, 2, E) * 0.25)
    for bias, group_top in ((b, 2), (None, 1), (b, 1)):
        check_route(P, logits_of(T, E, "bf16", 9, kind), 6, score=score, bias=bias, groups=8, top_groups=4,
                    group_top=group_top)
