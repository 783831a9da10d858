"""The expert-layer operators at the sizes they are used at: `run` takes a case through the
library (`own`) or through the same mathematics in elementary torch operations, `exact`
through 64-bit arithmetic, and `work` says what the case cannot do without.

  route    logits [T, E] -> the experts of each token and their weights
  matmul   y = x W^T with int8 weights (a scale for each output channel) and activations
           held in int8 (a scale for each token): quantised by the call, or given as int8
  experts  the routed experts' ReLU FFNs on such weights, weighted and summed for each token

A row r is held in 8 bits as q = the whole numbers nearest to r / s (ties to even) with the
32-bit scale s = max|r| / 127; an expert's activations h are 32-bit numbers that are held in
8 bits in the same way before the down product.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SMALLEST = 2.0 ** -100  # a row whose largest magnitude is below this is held as zeros


def listed():
    return [
        # one decoded token of a model with 64 experts: latency
        dict(name="route 1 token", op="route", T=1, E=64, k=8, score="softmax", dtype="f32",
             bias=False, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, masked=0.0),
        # a prefill chunk: sigmoid scores, a balancing bias, 4 of 8 groups
        dict(name="route grouped", op="route", T=4096, E=256, k=8, score="sigmoid", dtype="bf16",
             bias=True, groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, masked=0.0),
        # a long prompt, an odd number of tokens, experts that are switched off for some of
        # them (all of them for a few tokens), weights as the softmax leaves them
        dict(name="route long masked", op="route", T=30011, E=160, k=6, score="softmax",
             dtype="f16", bias=False, groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0,
             masked=0.1),
        # one decoded token through the up projection of the Llama-7B-shaped layer
        dict(name="matmul 1 token", op="matmul", M=1, K=4096, N=11008, x="f16", y="f16", bias=False),
        # a decode batch through its down projection
        dict(name="matmul 24 tokens", op="matmul", M=24, K=11008, N=4096, x="bf16", y="bf16",
             bias=False),
        # odd in every direction, 32-bit activations and outputs, a bias
        dict(name="matmul odd", op="matmul", M=333, K=1013, N=1101, x="f32", y="f32", bias=True),
        # a prefill chunk whose int8 activations several products share
        dict(name="matmul prefill", op="matmul", M=4096, K=4096, N=11008, x="i8", y="bf16",
             bias=False),
        # one decoded token through 2 of 8 experts of the Llama-7B shape
        dict(name="experts 1 token", op="experts", T=1, E=8, k=2, d=4096, f=11008, gated=True,
             x="f16", y="f16", bias=False, dropped=0.0),
        # a decode batch that reaches every expert
        dict(name="experts 16 tokens", op="experts", T=16, E=8, k=2, d=4096, f=11008, gated=True,
             x="f32", y="f32", bias=False, dropped=0.0),
        # many small experts, ragged counts, slots without an expert
        dict(name="experts fine", op="experts", T=777, E=64, k=6, d=2048, f=1408, gated=True,
             x="bf16", y="bf16", bias=False, dropped=0.1),
        # the plain ReLU form with its bias, odd widths
        dict(name="experts plain odd", op="experts", T=129, E=5, k=1, d=770, f=1999, gated=False,
             x="f32", y="f32", bias=True, dropped=0.0),
        # a prefill chunk through 2 of 8 experts of the Llama-7B shape
        dict(name="experts prefill", op="experts", T=4096, E=8, k=2, d=4096, f=11008, gated=True,
             x="bf16", y="bf16", bias=False, dropped=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "matmul", "experts"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * max(2, _log(rng, 8, 384) // groups)
        bias = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 30000), E=E, k=rng.randint(1, min(E, 12)),
                    score=rng.choice(("softmax", "sigmoid")), dtype=rng.choice(("f32", "f16", "bf16")),
                    bias=bias, groups=groups, top_groups=rng.randint(1, groups),
                    group_top=rng.choice((1, 2)), renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5)), masked=rng.choice((0.0, 0.0, 0.2)))
    if op == "matmul":
        x = rng.choice(("f32", "f16", "bf16", "i8"))
        return dict(op=op, M=_log(rng, 1, 4000), K=_log(rng, 64, 11000), N=_log(rng, 64, 11000), x=x,
                    y=rng.choice(("f32", "f16", "bf16")), bias=rng.random() < 0.3)
    E = _log(rng, 2, 64)
    k = rng.randint(1, min(E, 6))
    f = _log(rng, 100, 8000)
    d = min(_log(rng, 100, 4096), 600_000_000 // (3 * E * f))
    T = min(_log(rng, 1, 3000), 1_000_000_000_000 // (3 * k * d * f))
    x = rng.choice(("f32", "f16", "bf16"))
    return dict(op=op, T=T, E=E, k=k, d=d, f=f, gated=rng.random() < 0.7, x=x, y=x,
                bias=rng.random() < 0.3, dropped=rng.choice((0.0, 0.1)))


# ------------------------------------------------------------------------------- inputs
def _held(w):
    """Rows of 32-bit weights in 8 bits, in rows that begin at multiples of 16 bytes, and
    their scales."""
    a = w.abs().amax(-1)
    s = a / 127
    q = torch.round(w / s.unsqueeze(-1)).to(torch.int8)
    K = w.shape[-1]
    room = torch.zeros((*w.shape[:-1], (K + 15) // 16 * 16), dtype=torch.int8, device=w.device)
    room[..., :K] = q
    return room[..., :K], s


def _experts_held(gen, E, rows, K, dev):
    """[E, *rows, K] weights ~ N(0, 0.02) in 8 bits, an expert at a time."""
    room = torch.zeros((E, *rows, (K + 15) // 16 * 16), dtype=torch.int8, device=dev)
    scale = torch.empty((E, *rows), dtype=torch.float32, device=dev)
    for e in range(E):
        q, s = _held(torch.randn((*rows, K), generator=gen, device=dev) * 0.02)
        room[e, ..., :K] = q
        scale[e] = s
    return room[..., :K], scale


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rand = lambda *n: torch.randn(n, generator=gen, device=dev)  # noqa: E731
    st = dict(case)
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        # some experts are called more often than others
        l = rand(T, E) * 1.5 + rand(E) * 0.5
        if case["masked"]:
            l = torch.where(torch.rand((T, E), generator=gen, device=dev) < case["masked"], -math.inf, l)
            l[torch.rand(T, generator=gen, device=dev) < 0.01] = -math.inf
        st["logits"] = l.to(DTYPES[case["dtype"]])
        st["bias_t"] = rand(E) * 0.05 if case["bias"] else None
        return st
    if case["op"] == "matmul":
        M, K, N = case["M"], case["K"], case["N"]
        x = rand(M, K) * (0.5 + torch.rand((M, 1), generator=gen, device=dev))
        if case["x"] == "i8":
            st["xt"], st["xs"] = _held(x)
        else:
            st["xt"], st["xs"] = x.to(DTYPES[case["x"]]), None
        st["wq"], st["ws"] = _held(rand(N, K) * 0.02)
        st["bias_t"] = rand(N) if case["bias"] else None
        return st
    T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
    st["xt"] = rand(T, d).to(DTYPES[case["x"]])
    l = rand(T, E) + rand(E) * 0.5
    top = torch.topk(l, k, dim=1)
    idx = top.indices.to(torch.int32)
    if case["dropped"]:
        idx = torch.where(torch.rand((T, k), generator=gen, device=dev) < case["dropped"], -1, idx)
    st["idx"], st["weights"] = idx.contiguous(), torch.softmax(top.values, 1).contiguous()
    st["wa"], st["sa"] = _experts_held(gen, E, (f, 2) if case["gated"] else (f,), d, dev)
    st["wd"], st["sd"] = _experts_held(gen, E, (d,), f, dev)
    st["bias_t"] = rand(E, f) * 0.3 - 0.5 if case["bias"] else None
    return st


# ----------------------------------------------------------------------------- plain forms
def _route(l, k, score, bias, groups, top_groups, group_top, renorm, scale):
    # 64 bits: the choice of an expert is a comparison, and two scores may lie next to each other
    l = l.double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    T, E = l.shape
    on = l > -math.inf
    if score == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.where(on, torch.where(l == m, 1.0, torch.exp(l - m)), 0.0)
        s = e / e.sum(1, keepdim=True).clamp_min(1.0)  # at least 1 where any expert is on
    else:
        s = 1 / (1 + torch.exp(-l))
    # without a bias the scores are in the order of the logits
    c = l if bias is None else s + bias.double()
    c = torch.where(on & ~torch.isnan(c), c, -math.inf)
    if groups > 1:
        v = c if group_top == 1 or bias is not None else torch.where(on, s, -math.inf)
        v = torch.sort(v.reshape(T, groups, E // groups), dim=2, descending=True).values
        g = v[:, :, 0]
        if group_top == 2 and E // groups > 1:
            g = g + torch.where(v[:, :, 1] > -math.inf, v[:, :, 1], 0.0)
        order = torch.sort(g, dim=1, descending=True, stable=True).indices[:, :top_groups]
        kept = torch.zeros_like(g, dtype=torch.bool).scatter_(1, order, True)
        c = torch.where(kept.repeat_interleave(E // groups, 1), c, -math.inf)
    c, idx = torch.sort(c, dim=1, descending=True, stable=True)
    c, idx = c[:, :k], idx[:, :k]
    none = c == -math.inf
    w = torch.where(none, 0.0, s.gather(1, idx))
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(none, -1, idx).to(torch.int32), (w * scale).float()


def _quantize(x):
    """Rows of 32-bit numbers as the whole numbers of 8 bits that they are held as, in 32
    bits, and the scales."""
    a = x.abs().amax(1)
    s = torch.where(a < SMALLEST, 0.0, a / 127)
    # 64 bits: x / s may lie next to a border between two whole numbers
    q = torch.round(x.double() / s.double().unsqueeze(1))
    return torch.where(s.unsqueeze(1) > 0, q, 0.0).float(), s


def _matmul(x, xs, wq, ws, bias, out):
    q, s = (x.float(), xs) if xs is not None else _quantize(x.float())
    # the sums of products are whole numbers: exact in 32 bits up to 2^24
    y = (q @ wq.float().t()) * (s.unsqueeze(1) * ws)
    return (y if bias is None else y + bias).to(out)


def _experts(x, idx, weights, wa, sa, wd, sd, bias, out):
    T, d = x.shape
    E, f, k = wa.shape[0], wa.shape[1], idx.shape[1]
    on = (idx >= 0) & (idx < E)
    at = torch.where(on, idx, 0).long()
    q, s = _quantize(x.float())
    slot = torch.arange(T, device=x.device).unsqueeze(1)
    a = (q @ wa.reshape(-1, d).float().t()).reshape(T, E, -1)[slot, at]  # [T, k, rows]
    # 64 bits up to the one rounding of h: it decides between two whole numbers afterwards
    a = a.double() * (s.double().reshape(T, 1, 1) * sa.reshape(E, -1)[at].double())
    if wa.dim() == 4:
        a = a.reshape(T, k, f, 2)
        g, u = a[..., 0], a[..., 1]
    else:
        g, u = a, None
    if bias is not None:
        g = g + bias[at].double()
    h = torch.relu(g)
    h = (h if u is None else h * u).float().reshape(T * k, f)
    hq, hs = _quantize(h)
    p = (hq @ wd.reshape(-1, f).float().t()).reshape(T, k, E, d)
    p = p.gather(2, at.reshape(T, k, 1, 1).expand(T, k, 1, d)).squeeze(2)
    p = p * (hs.reshape(T, k, 1) * sd[at])
    return torch.where(on.unsqueeze(2), weights.unsqueeze(2) * p, 0.0).sum(1).to(out)


def run(st):
    op = st["op"]
    if own:
        import activation_sparse_decode_rank_amd as lib

        if op == "route":
            return lib.route(st["logits"], st["k"], score=st["score"], bias=st["bias_t"],
                             groups=st["groups"], top_groups=st["top_groups"],
                             group_top=st["group_top"], renormalize=st["renorm"], scale=st["scale"])
        if op == "matmul":
            return lib.i8_matmul(st["xt"], st["wq"], st["ws"], x_scale=st["xs"], bias=st["bias_t"],
                                 out_dtype=DTYPES[st["y"]])
        return lib.experts(st["xt"], st["idx"], st["weights"], st["wa"], st["sa"], st["wd"], st["sd"],
                           b_act=st["bias_t"], out_dtype=DTYPES[st["y"]])
    if op == "route":
        return _route(st["logits"], st["k"], st["score"], st["bias_t"], st["groups"], st["top_groups"],
                      st["group_top"], st["renorm"], st["scale"])
    if op == "matmul":
        return _matmul(st["xt"], st["xs"], st["wq"], st["ws"], st["bias_t"], DTYPES[st["y"]])
    return _experts(st["xt"], st["idx"], st["weights"], st["wa"], st["sa"], st["wd"], st["sd"],
                    st["bias_t"], DTYPES[st["y"]])


# ------------------------------------------------------------------------------------ work
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # an exponential and a few comparisons for each expert, k comparisons of each
        return {"bytes": T * E * SIZE[case["dtype"]] + T * k * 8 + (4 * E if case["bias"] else 0),
                "flops": T * E * (8 + k)}
    if case["op"] == "matmul":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * K * SIZE[case["x"]] + N * K + 4 * N + M * N * SIZE[case["y"]]
                + (4 * M if case["x"] == "i8" else 0) + (4 * N if case["bias"] else 0),
                "flops": 2 * M * K * N}
    T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
    m = 3 if case["gated"] else 2
    rows = T * k * (1 - case["dropped"])
    # the experts that these rows are expected to reach
    reached = E * (1 - (1 - 1 / E) ** rows)
    return {"bytes": reached * (m * d * f + 4 * (m - 1) * f + 4 * d)
            + T * d * (SIZE[case["x"]] + SIZE[case["y"]]) + 8 * T * k,
            "flops": 2 * rows * m * d * f}


# --------------------------------------------------------------------------- 64-bit values
def _exact_route(case, st):
    l = st["logits"].float().cpu().numpy().astype(np.float64)
    bias = None if st["bias_t"] is None else st["bias_t"].cpu().numpy().astype(np.float64)
    T, E = l.shape
    k, G = case["k"], case["groups"]
    per = E // G
    off = ~(l > -np.inf)  # minus infinity and NaN: the expert is off
    with np.errstate(all="ignore"):
        if case["score"] == "sigmoid":
            s = np.exp(-np.logaddexp(0.0, -l))
        else:
            top = np.max(np.where(off, -np.inf, l), axis=1)
            e = np.where(off, 0.0, np.exp(np.where(off, 0.0, l - top[:, None])))
            s = e / np.maximum(e.sum(axis=1), 1.0)[:, None]
    c = l.copy() if bias is None else s + bias
    c[off] = -np.inf
    if G > 1:
        v = np.where(off, -np.inf, s) if bias is None and case["group_top"] == 2 else c
        v = -np.sort(-v.reshape(T, G, per), axis=2)
        g = v[:, :, 0].copy()
        if case["group_top"] == 2 and per > 1:
            more = v[:, :, 1]
            g = g + np.where(np.isneginf(more), 0.0, more)
        first = np.argsort(-g, axis=1, kind="stable")[:, :case["top_groups"]]
        keep = np.zeros((T, G), bool)
        np.put_along_axis(keep, first, True, axis=1)
        c[~np.repeat(keep, per, axis=1)] = -np.inf
    idx = np.argsort(-c, axis=1, kind="stable")[:, :k]
    none = np.isneginf(np.take_along_axis(c, idx, 1))
    w = np.where(none, 0.0, np.take_along_axis(s, idx, 1))
    if case["renorm"]:
        t = w.sum(axis=1, keepdims=True)
        w = np.divide(w, t, out=np.zeros_like(w), where=t > 0)
    return [np.where(none, -1, idx).astype(np.int32), w * case["scale"]]


def _exact_rows(v):
    """64-bit rows (each value a 32-bit number) -> whole numbers and scales in 64 bits; the
    scale is a 32-bit number by definition."""
    big = v.abs().max(dim=1).values
    s = (big / 127).float().double()
    s[big < SMALLEST] = 0
    q = torch.zeros_like(v)
    rows = s > 0
    q[rows] = torch.round(v[rows] / s[rows, None])
    return q, s


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, st)
    x = st["xt"].double()
    if case["op"] == "matmul":
        q, s = (x, st["xs"].double()) if case["x"] == "i8" else _exact_rows(x)
        y = torch.matmul(q, st["wq"].double().t().contiguous())
        y *= s[:, None]
        y *= st["ws"].double()[None]
        if st["bias_t"] is not None:
            y += st["bias_t"].double()
        return y
    q, s = _exact_rows(x)
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        t, slot = torch.nonzero(st["idx"] == e, as_tuple=True)
        if not t.numel():
            continue
        wa, sa = st["wa"][e].double(), st["sa"][e].double()
        m = 2 if case["gated"] else 1
        acts = [torch.matmul(q[t], wa.reshape(-1, m, case["d"])[:, j].t().contiguous())
                * sa.reshape(-1, m)[:, j] * s[t, None] for j in range(m)]
        h = acts[0] if st["bias_t"] is None else acts[0] + st["bias_t"][e].double()
        h = h * (h > 0)
        if m == 2:
            h = h * acts[1]
        hq, hs = _exact_rows(h.float().double())
        part = torch.matmul(hq, st["wd"][e].double().t().contiguous()) * st["sd"][e].double() * hs[:, None]
        y.index_add_(0, t, part * st["weights"][t, slot].double()[:, None])
    return y
