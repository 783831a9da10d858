"""CPU tests of include/sparse_ffn_experts.h: it compiles as C, the library exports what it
declares, the ctypes mirror has the C layout, every refusal happens on the host, and the
scratch plan (csrc/sffn_i8_host.h) covers what the calls carve out of it."""
import ctypes as C
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sparse_ffn_experts.h")
A = 0x10000  # an aligned address that is never dereferenced: the calls refuse first


@pytest.fixture(scope="module")
def N():
    from activation_sparse_decode_rank_amd import _native
    return _native


def test_header_compiles_as_c_and_is_exported(N):
    src = ('#include "sparse_ffn_experts.h"\n'
           'int main(void){ sffn_experts_desc d; (void)d; return SFFN_BF16; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I",
                        os.path.dirname(HEADER), "-x", "c", "-"], input=src, text=True,
                       capture_output=True)
    assert r.returncode == 0, r.stderr
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sparse_ffn_\w+)\s*\(", text)))
    assert set(names) == set(N.EXPORTED_EXPERTS)
    out = subprocess.run(["nm", "-D", "--defined-only", N.LIB_PATH], capture_output=True,
                         text=True).stdout
    for name in names:
        assert re.search(rf"\bT {name}\b", out), name


def test_desc_layout_and_constants_match_header(N, tmp_path):
    D = N.SffnExpertsDesc
    fields = [f[0] for f in D._fields_]
    src = ('#include <stddef.h>\n#include <stdio.h>\n#include "sparse_ffn_experts.h"\n'
           'int main(void){ printf("%zu %d %d %d %d %d", sizeof(sffn_experts_desc), SFFN_BF16, SFFN_I8, '
           'SFFN_MAX_EXPERTS, SFFN_MAX_TOPK, SFFN_I8_MAX_K);\n'
           + "".join(f'printf(" %zu", offsetof(sffn_experts_desc, {f}));\n' for f in fields)
           + "return 0; }\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), "-x", "c", "-", "-o", exe],
                   input=src, text=True, check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(D), N.SFFN_BF16, N.SFFN_I8, N.SFFN_MAX_EXPERTS, N.SFFN_MAX_TOPK,
                   N.SFFN_I8_MAX_K] + [getattr(D, f).offset for f in fields]


def route(N, **over):
    a = dict(logits=A, dtype=0, ld=64, T=4, E=64, k=8, score=0, bias=None, groups=1, top_groups=1,
             group_top=1, renorm=1, scale=1.0, idx=A, weights=A, stream=None)
    a.update(over)
    return N.lib().sparse_ffn_route(*a.values())


@pytest.mark.parametrize("over", [
    dict(logits=None), dict(idx=None), dict(weights=None), dict(dtype=3), dict(dtype=-1), dict(T=-1),
    dict(E=0), dict(k=0), dict(k=65), dict(ld=63), dict(score=2), dict(groups=0), dict(groups=3),
    dict(groups=8, top_groups=9), dict(groups=8, top_groups=0), dict(group_top=0),
    dict(group_top=3), dict(renorm=2), dict(logits=A + 2), dict(bias=A + 1), dict(idx=A + 2),
])
def test_route_refuses(N, over):
    assert route(N, **over) == N.SFFN_ERR_INVALID


@pytest.mark.parametrize("over", [
    dict(E=1025, ld=1025), dict(E=256, ld=256, k=65), dict(E=256, ld=256, groups=128),
])
def test_route_unsupported(N, over):
    assert route(N, **over) == N.SFFN_ERR_UNSUPPORTED


def test_no_tokens_is_fine(N):
    L = N.lib()
    assert route(N, T=0, logits=None, idx=None, weights=None) == N.SFFN_OK
    assert L.sparse_ffn_quantize_rows(None, 0, 8, 0, 8, None, 16, None, None) == N.SFFN_OK
    assert L.sparse_ffn_i8_matmul(None, 0, None, 8, 0, 8, None, 16, None, None, 4, None, 0, 4, None,
                                  0, None) == N.SFFN_OK
    D = desc(N)
    assert L.sparse_ffn_experts(C.byref(D), None, 0, 64, 0, None, None, 2, None, 0, 64, None, 0,
                                None) == N.SFFN_OK


@pytest.mark.parametrize("over", [
    dict(x=None), dict(q=None), dict(scale=None), dict(dtype=3), dict(dtype=7), dict(rows=-1),
    dict(cols=0), dict(ldx=32), dict(ldq=47), dict(ldq=32), dict(q=A + 8), dict(x=A + 2),
    dict(scale=A + 2),
])
def test_quantize_refuses(N, over):
    a = dict(x=A, dtype=0, ldx=33, rows=4, cols=33, q=A, ldq=48, scale=A, stream=None)
    a.update(over)
    assert N.lib().sparse_ffn_quantize_rows(*a.values()) == N.SFFN_ERR_INVALID


def matmul(lib, **over):
    a = dict(x=A, xd=1, xs=None, ldx=100, M=5, K=100, w=A, ldw=112, ws=A, bias=None, N=7, y=A, yd=0,
             ldy=7, work=A, work_bytes=1 << 20, stream=None)
    a.update(over)
    return lib.lib().sparse_ffn_i8_matmul(*a.values())


@pytest.mark.parametrize("over", [
    dict(x=None), dict(w=None), dict(ws=None), dict(y=None), dict(xd=4), dict(yd=3), dict(M=-1),
    dict(K=0), dict(N=0), dict(ldx=99), dict(ldy=6), dict(ldw=100), dict(ldw=96), dict(w=A + 8),
    dict(x=A + 1), dict(y=A + 2), dict(xs=A), dict(xd=3), dict(work=None), dict(work=A + 16),
    dict(work_bytes=16), dict(bias=A + 2),
])
def test_matmul_refuses(N, over):
    assert matmul(N, **over) == N.SFFN_ERR_INVALID


def test_matmul_unsupported(N):
    K = N.SFFN_I8_MAX_K + 1
    assert matmul(N, K=K, ldx=K, ldw=K + 16) == N.SFFN_ERR_UNSUPPORTED
    assert matmul(N, ldw=(1 << 24) + 16) == N.SFFN_ERR_UNSUPPORTED
    assert experts(N, desc(N, ld_act=(1 << 24) + 16)) == N.SFFN_ERR_UNSUPPORTED
    assert experts(N, desc(N, ld_down=1 << 40)) == N.SFFN_ERR_UNSUPPORTED
    n = (1 << 31) - 1
    assert matmul(N, M=n) == N.SFFN_ERR_UNSUPPORTED
    assert matmul(N, M=n, N=n, ldy=n) == N.SFFN_ERR_UNSUPPORTED
    wb = N.sparse_ffn_i8_matmul_work_bytes
    none = C.c_size_t(-1).value
    assert wb(0, 4, 4, K) == none and wb(9, 4, 4, 64) == none and wb(0, -1, 4, 64) == none
    assert wb(0, 0, 4, 64) == 0


def desc(N, **over):
    D = N.SffnExpertsDesc()
    D.experts, D.d, D.d_ffn, D.gated = 4, 64, 100, 1
    D.w_act, D.ld_act, D.act_scale = A, 64, A
    D.w_down, D.ld_down, D.down_scale = A, 112, A
    for k, v in over.items():
        setattr(D, k, v)
    return D


def experts(N, D, **over):
    a = dict(x=A, xd=0, ldx=64, T=3, idx=A, weights=A, k=2, y=A, yd=0, ldy=64, work=A,
             work_bytes=1 << 24, stream=None)
    a.update(over)
    return N.lib().sparse_ffn_experts(None if D is None else C.byref(D), *a.values())


@pytest.mark.parametrize("over", [
    dict(experts=0), dict(d=0), dict(d_ffn=-1), dict(gated=2), dict(w_act=None), dict(w_down=None),
    dict(act_scale=None), dict(down_scale=None), dict(ld_act=48), dict(ld_act=72),
    dict(ld_down=100), dict(ld_down=96), dict(w_act=A + 4), dict(w_down=A + 8), dict(b_act=A + 2),
])
def test_experts_desc_refused(N, over):
    assert experts(N, desc(N, **over)) == N.SFFN_ERR_INVALID


@pytest.mark.parametrize("over", [
    dict(x=None), dict(idx=None), dict(weights=None), dict(y=None), dict(xd=3), dict(yd=3),
    dict(T=-1), dict(k=0), dict(ldx=63), dict(ldy=63), dict(work=None), dict(work=A + 64),
    dict(work_bytes=64), dict(idx=A + 2), dict(x=A + 2),
])
def test_experts_refuses(N, over):
    assert experts(N, desc(N), **over) == N.SFFN_ERR_INVALID


def test_experts_unsupported(N):
    assert experts(N, desc(N), k=65) == N.SFFN_ERR_UNSUPPORTED
    assert experts(N, desc(N, experts=1025)) == N.SFFN_ERR_UNSUPPORTED
    assert experts(N, desc(N, d_ffn=1 << 20, ld_down=1 << 20)) == N.SFFN_ERR_UNSUPPORTED
    assert experts(N, None) == N.SFFN_ERR_INVALID
    assert N.sparse_ffn_experts_work_bytes(desc(N, d=0), 4, 2) == 0
    assert N.sparse_ffn_experts_work_bytes(desc(N), 0, 2) == 0
    assert N.sparse_ffn_experts_work_bytes(desc(N), 4, 65) == 0


def test_scratch_plan(tmp_path):
    """Regions follow each other without overlap, the chunk is the most tokens that fit, and a
    tile table never needs more entries than it has."""
    src = r'''
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "sffn_i8_host.h"
using namespace sffn::host;
#define CHECK(c) do { if (!(c)) { std::printf("failed: %s line %d\n", #c, __LINE__); std::exit(1); } } while (0)
int main() {
  std::mt19937 g(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(g() % (unsigned)(hi - lo + 1)); };
  for (int it = 0; it < 3000; ++it) {
    const int E = pick(1, it % 3 ? 64 : 1024), d = pick(1, 5000), f = pick(1, 12000);
    const int k = pick(1, 64), T = pick(1, it % 2 ? 300 : 20000);
    const ExpertsCarve c = experts_carve(E, d, f, T, k);
    const size_t R = (size_t)T * k;
    const size_t at[] = {c.xq, c.xs, c.offs, c.src, c.tiles, c.count, c.h, c.hq, c.hs, c.part, c.bytes};
    const size_t need[] = {(size_t)T * i8_kpad(d), (size_t)T * 4, ((size_t)E + 1) * 4, R * 4,
                           (size_t)c.max_tiles * 8, 4, R * c.ldh * 4, R * (size_t)i8_kpad(f), R * 4,
                           R * c.ldp * 4};
    for (int i = 0; i < 10; ++i) { CHECK(at[i] % 256 == 0); CHECK(at[i] + need[i] <= at[i + 1]); }
    CHECK(c.ldh >= (size_t)f && c.ldp >= (size_t)d && i8_kpad(d) >= d && i8_kpad(d) % 256 == 0);
    // any split of the rows over the experts
    std::vector<size_t> n(E, 0);
    const int used = pick(1, E);
    for (size_t r = 0; r < std::min<size_t>(R, 4000); ++r) n[g() % used]++;
    size_t tiles = 0, rows = 0;
    for (size_t v : n) { tiles += (v + c.tile - 1) / c.tile; rows += v; }
    if (rows == R) CHECK(tiles <= (size_t)c.max_tiles);
    const size_t some = c.bytes / (size_t)pick(1, 9) + 1;
    const int ch = experts_chunk(E, d, f, T, k, some);
    CHECK(ch <= T && (size_t)ch * k <= kExpertsMaxRows);
    if (ch > 0) CHECK(experts_carve(E, d, f, ch, k).bytes <= some);
    if (ch < T && (size_t)(ch + 1) * k <= kExpertsMaxRows) CHECK(experts_carve(E, d, f, ch + 1, k).bytes > some);
    const I8MatmulCarve m = i8_matmul_carve(T, d);
    CHECK((size_t)T * i8_kpad(d) <= m.scale && m.scale + (size_t)T * 4 <= m.bytes);
  }
  CHECK(experts_chunk(8, 64, 64, 100, 2, 0) == 0);
  std::puts("ok");
  return 0;
}
'''
    (tmp_path / "plan.cpp").write_text(src)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I",
                    os.path.join(ROOT, "activation_sparse_decode_rank_amd", "csrc"),
                    str(tmp_path / "plan.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout


def test_python_calls_want_device_tensors():
    import torch
    import activation_sparse_decode_rank_amd as P
    x = torch.zeros((2, 16))
    q, s = torch.zeros((4, 16), dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError):
        P.route(x, 2)
    with pytest.raises(ValueError):
        P.quantize_rows(x)
    with pytest.raises(ValueError):
        P.i8_matmul(x, q, s)
    with pytest.raises(ValueError):
        P.ExpertFFN(w_act=q, act_scale=s, w_down=q, down_scale=s)
