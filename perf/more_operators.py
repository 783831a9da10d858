"""The operators in front of a layer's products and with 4-bit weights, at the sizes they are
used at: `run` takes a case through the library (`own`) or through the same mathematics in
elementary torch operations, `exact` through 64-bit arithmetic, and `work` says what the case
cannot do without.

  norm      y = v w / sqrt(mean(v^2) + eps) with v = x, or x + residual rounded to x's type
            (returned too): float rows, rows held in 8 bits, or rows in 4-bit blocks
  quantize  rows into 4-bit blocks, and the values that they stand for
  matmul    y = x W^T with W in 4-bit blocks and x in 4-bit blocks: made so by the call, or given so

A row in 4-bit blocks: 32 neighbours share a scale 2^e, the power of two with
3.5 2^e <= max|r| < 7 2^e, held as the byte e + 127; each is held as the number of 0, 0.5, 1,
1.5, 2, 3, 4, 6 and their negatives that is nearest to r / 2^e (ties to the even code). A row
r is held in 8 bits as the whole numbers nearest to r / s (ties to even) with the 32-bit scale
s = max|r| * fl(1 / 127). What is held in 8 or 4 bits is returned as the values it stands for.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    return [
        # one decoded token in front of a Llama-7B-shaped FFN with 8-bit weights: latency
        dict(name="norm 1 token", op="norm", T=1, d=4096, x="f16", residual=True, out="i8"),
        # odd in both directions, 32-bit rows, no residual
        dict(name="norm odd", op="norm", T=333, d=1013, x="f32", residual=False, out="f32"),
        # a prefill chunk into 8 bits
        dict(name="norm prefill", op="norm", T=4096, d=4096, x="bf16", residual=True, out="i8"),
        # a prefill chunk of the OPT-175B width into 4-bit blocks
        dict(name="norm wide", op="norm", T=2048, d=12288, x="bf16", residual=True, out="mx4"),
        # activations of an odd length, as a prompt's tokens come
        dict(name="quantize odd", op="quantize", R=777, K=1999, x="bf16"),
        # a weight matrix of the Llama-7B shape
        dict(name="quantize weights", op="quantize", R=11008, K=4096, x="f32"),
        # one decoded token through the up projection of the Llama-7B-shaped layer
        dict(name="matmul 1 token", op="matmul", M=1, K=4096, N=11008, x="f16", y="f16", bias=False),
        # one decoded token through the up projection of the OPT-175B-shaped layer
        dict(name="matmul 1 token wide", op="matmul", M=1, K=12288, N=49152, x="f32", y="f32",
             bias=True),
        # a decode batch through the down projection of the Llama-7B-shaped layer
        dict(name="matmul 24 tokens", op="matmul", M=24, K=11008, N=4096, x="bf16", y="bf16",
             bias=False),
        # odd in every direction, 32-bit activations and outputs, a bias
        dict(name="matmul odd", op="matmul", M=333, K=1013, N=1101, x="f32", y="f32", bias=True),
        # a prefill chunk whose 4-bit activations several products share
        dict(name="matmul prefill", op="matmul", M=4096, K=4096, N=11008, x="mx4", y="bf16",
             bias=False),
        # a prompt through the OPT-175B-shaped up projection
        dict(name="matmul prompt wide", op="matmul", M=512, K=12288, N=49152, x="bf16", y="bf16",
             bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "quantize", "matmul", "matmul", "matmul"))
    x = rng.choice(("f32", "f16", "bf16"))
    if op == "norm":
        T, d = _log(rng, 1, 4096), _log(rng, 64, 12288)
        return dict(op=op, T=T, d=d, x=x, residual=rng.random() < 0.6,
                    out=rng.choice(("i8", "i8", "mx4", x)))
    if op == "quantize":
        return dict(op=op, R=_log(rng, 1, 11008), K=_log(rng, 33, 4096), x=x)
    M, K, N = _log(rng, 1, 4000), _log(rng, 64, 12000), _log(rng, 64, 12000)
    return dict(op=op, M=M, K=K, N=N, x=rng.choice((x, x, "mx4")), y=rng.choice(("f32", "f16", "bf16")),
                bias=rng.random() < 0.3)


# ------------------------------------------------------------------------------- inputs
def _packed(values, e):
    """Values on the 4-bit grid [R, B, 32] and exponents [R, B] as bytes: two codes a byte, the
    first in the low half, and e + 127 in rows that begin at multiples of 16 bytes."""
    R, B, _ = values.shape
    a = values.abs()
    # the codes 0 .. 7 are the grid in order: twice the value below 2, value + 2, value / 2 + 4
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code += 8 * torch.signbit(values).to(torch.uint8)
    code = code.reshape(R, -1, 2)
    room = torch.zeros((R, (B + 15) // 16 * 16), dtype=torch.uint8, device=values.device)
    room[:, :B] = (e + 127).to(torch.uint8)
    return code[..., 0] + 16 * code[..., 1], room[:, :B]


def _held4(x):
    """Rows of 32-bit numbers packed, some hundred megabytes of them at a time."""
    R, K = x.shape
    step = max(1, (1 << 26) // K)
    parts = []
    for r in range(0, R, step):
        v, e = _blocks(x[r:r + step])
        parts.append(_packed(v, e))
    q = torch.cat([p[0] for p in parts])
    room = torch.zeros((R, (parts[0][1].shape[1] + 15) // 16 * 16), dtype=torch.uint8, device=x.device)
    s = room[:, :parts[0][1].shape[1]]
    s.copy_(torch.cat([p[1] for p in parts]))
    return q, s


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rand = lambda *n: torch.randn(n, generator=gen, device=dev)  # noqa: E731
    st = dict(case)
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        dt = DTYPES[case["x"]]
        # a residual stream grows larger than what a layer adds, in some channels much larger
        far = torch.where(torch.rand(d, generator=gen, device=dev) < 0.01, 20.0, 1.0)
        st["xt"] = (rand(T, d) * (1.0 if case["residual"] else far)).to(dt)
        st["res"] = (rand(T, d) * 3 * far).to(dt) if case["residual"] else None
        st["w"] = (1 + 0.2 * rand(d)).to(dt)
        return st
    if case["op"] == "quantize":
        st["xt"] = (rand(case["R"], case["K"]) * 0.02).to(DTYPES[case["x"]])
        return st
    M, K, N = case["M"], case["K"], case["N"]
    x = rand(M, K) * (0.5 + torch.rand((M, 1), generator=gen, device=dev))
    if case["x"] == "mx4":
        st["xt"], st["xs"] = _held4(x)
    else:
        st["xt"], st["xs"] = x.to(DTYPES[case["x"]]), None
    st["wq"], st["ws"] = _held4(rand(N, K).mul_(0.02))
    st["bias_t"] = rand(N) if case["bias"] else None
    return st


# ----------------------------------------------------------------------------- plain forms
def _blocks(x):
    """Rows of 32-bit numbers in blocks of 32: the numbers of the 4-bit grid [R, B, 32] and the
    exponents of the scales [R, B]."""
    R, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 32)).reshape(R, -1, 32)
    m, e = torch.frexp(x.abs().amax(2))  # m in [0.5, 1)
    e = torch.where(m == 0, -127, (e - 3 + (m >= 0.875).int()).clamp_min(-127))
    # 64 bits: the scale may lie below the smallest normal number of 32
    t = torch.ldexp(x.double(), -e.unsqueeze(2)).float()
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, t), e


def _unpacked(q, s):
    """The 32-bit values of packed rows."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=q.device)
    v = torch.stack((grid[(q & 15).int()], grid[(q >> 4).int()]), 2)
    v = v.reshape(q.shape[0], -1, 32) * torch.ldexp(torch.ones((), device=q.device),
                                                    s.int() - 127).unsqueeze(2)
    return v.reshape(q.shape[0], -1)


def _values4(x):
    v, e = _blocks(x)
    return (v * torch.ldexp(torch.ones((), device=x.device), e).unsqueeze(2)).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _norm(x, w, res, out):
    v = x if res is None else x + res
    if out in DTYPES:
        f = v.float()
        y = f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * w.float()
        return [y.to(DTYPES[out])] + ([] if res is None else [v])
    # 64 bits up to the one rounding of the row: it decides between two held numbers afterwards
    f = v.double()
    y = (f * w.double() / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)).float()
    if out == "mx4":
        y = _values4(y).to(x.dtype)
    else:
        s = y.abs().amax(1, keepdim=True) * (1 / 127)
        q = torch.round(y.double() / s.double()).float()  # 64 bits: y / s may lie next to a border
        y = q * s
    return [y] + ([] if res is None else [v])


def _matmul(x, xs, w, ws, bias, out):
    x = _values4(x.float()) if xs is None else _unpacked(x, xs)
    y = x @ _unpacked(w, ws)[:, :x.shape[1]].t()
    return (y if bias is None else y + bias).to(out)


def run(st):
    op = st["op"]
    if own:
        import activation_sparse_decode_rank_amd as lib

        if op == "norm":
            out = st["out"]
            got = lib.rms_norm(st["xt"], st["w"], residual=st["res"], eps=EPS,
                               out=DTYPES.get(out, out))
            if out in DTYPES:
                return [got] if st["res"] is None else list(got)
            if out == "mx4":
                y = lib.dequantize_mx4(got[0], got[1], cols=st["d"], dtype=st["xt"].dtype)
            else:
                y = got[0] * got[1].unsqueeze(1)
            return [y] + list(got[2:])
        if op == "quantize":
            q, s = lib.quantize_mx4(st["xt"])
            return lib.dequantize_mx4(q, s, cols=st["K"], dtype=st["xt"].dtype)
        return lib.mx4_matmul(st["xt"], st["wq"], st["ws"], x_scale=st["xs"], bias=st["bias_t"],
                              out_dtype=DTYPES[st["y"]])
    if op == "norm":
        return _norm(st["xt"], st["w"], st["res"], st["out"])
    if op == "quantize":
        return _values4(st["xt"].float()).to(st["xt"].dtype)
    return _matmul(st["xt"], st["xs"], st["wq"], st["ws"], st["bias_t"], DTYPES[st["y"]])


# ------------------------------------------------------------------------------------ work
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1, "mx4": 17 / 32}


def work(case):
    if case["op"] == "norm":
        n, out = case["T"] * case["d"], case["out"]
        # what is held in 8 or 4 bits is written, and the values that it stands for
        y = SIZE[out] if out in DTYPES else SIZE[out] + (4 if out == "i8" else SIZE[case["x"]])
        return {"bytes": n * ((3 if case["residual"] else 1) * SIZE[case["x"]] + y) + case["d"] * SIZE[case["x"]],
                "flops": n * (8 if case["residual"] else 7)}
    if case["op"] == "quantize":
        n = case["R"] * case["K"]
        return {"bytes": n * (2 * SIZE[case["x"]] + SIZE["mx4"]), "flops": n * 4}
    M, K, N = case["M"], case["K"], case["N"]
    return {"bytes": M * K * SIZE[case["x"]] + N * K * SIZE["mx4"] + M * N * SIZE[case["y"]]
            + (4 * N if case["bias"] else 0),
            "flops": 2 * M * K * N}


# --------------------------------------------------------------------------- 64-bit values
def _exact4(v):
    """64-bit rows -> the values that they are held as in 4-bit blocks."""
    R, K = v.shape
    out = torch.zeros((R, (K + 31) // 32 * 32), dtype=torch.float64, device=v.device)
    out[:, :K] = v
    out = out.view(R, -1, 32)
    big = out.abs().max(dim=2).values
    e = torch.ceil(torch.log2(torch.where(big > 0, big, 1.0) / 7))
    e = e + (big >= 7 * torch.exp2(e)).double()
    e = e - (big < 7 * torch.exp2(e - 1)).double()
    s = torch.exp2(torch.clamp(torch.where(big > 0, e, -127.0), min=-127.0))[..., None]
    grid = torch.tensor(GRID, dtype=torch.float64, device=v.device)
    middle = (grid[1:] + grid[:-1]) / 2
    a = (out.abs() / s).contiguous()
    low, high = torch.bucketize(a, middle), torch.bucketize(a, middle, right=True)
    out = torch.sign(out) * grid[torch.where(low % 2 == 0, low, high)] * s
    return out.reshape(R, -1)[:, :K]


def _decoded(q, s):
    """64-bit values of packed rows, from the fields of their codes: sign, two bits of exponent,
    one of mantissa."""
    R, n = q.shape
    out = torch.empty((R, 2 * n), dtype=torch.float64, device=q.device)
    for half in range(2):
        c = torch.bitwise_and(torch.bitwise_right_shift(q, 4 * half), 15)
        exp, man = ((c >> 1) & 3).double(), (c & 1).double()
        v = torch.where(exp > 0, (1 + man / 2) * torch.exp2(exp - 1), man / 2)
        out[:, half::2] = torch.where(c >= 8, -v, v)
    return (out.view(R, -1, 32) * torch.exp2(s.double() - 127)[..., None]).view(R, -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact4(st["xt"].double())
    if case["op"] == "matmul":
        x = st["xt"]
        M = x.shape[0]
        x = _decoded(x, st["xs"]) if case["x"] == "mx4" else _exact4(x.double())
        y = torch.empty((M, case["N"]), dtype=torch.float64, device=x.device)
        step = max(1, (1 << 28) // case["K"])
        for n in range(0, case["N"], step):
            w = _decoded(st["wq"][n:n + step], st["ws"][n:n + step])[:, :x.shape[1]]
            y[:, n:n + step] = torch.matmul(x, w.t().contiguous())
        if st["bias_t"] is not None:
            y += st["bias_t"].double()
        return y
    x = st["xt"].cpu().double().numpy()
    if case["residual"]:
        x = torch.from_numpy(x + st["res"].cpu().double().numpy()).to(st["xt"].dtype).double().numpy()
    v = [] if not case["residual"] else [x]
    ms = np.einsum("td,td->t", x, x) / case["d"]
    y = x / np.sqrt(ms + EPS)[:, None] * st["w"].cpu().double().numpy()
    if case["out"] in DTYPES:
        return [y] + v
    y = y.astype(np.float32).astype(np.float64)
    if case["out"] == "mx4":
        return [_exact4(torch.from_numpy(y).to(st["xt"].device))] + v
    s = np.abs(y).max(axis=1).astype(np.float32) * (np.float32(1) / np.float32(127))
    s = s.astype(np.float64)[:, None]
    return [np.rint(y / s) * s] + v
