"""CPU tests of include/sparse_ffn_mx4.h: it compiles as C, the library exports what it declares,
every refusal happens on the host, the Python calls refuse what they cannot pass on, and the
scratch plan (csrc/sffn_mx4_host.h) covers what a call carves out of it."""
import ctypes as C
import math
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sparse_ffn_mx4.h")
A = 0x10000  # an aligned address that is never dereferenced: the calls refuse first


@pytest.fixture(scope="module")
def N():
    from activation_sparse_decode_rank_amd import _native
    return _native


def test_header_compiles_as_c_and_is_exported(N, tmp_path):
    src = ('#include <stdio.h>\n#include "sparse_ffn_mx4.h"\n'
           'int main(void){ printf("%d %d", SFFN_MX4, SFFN_MX4_MAX_K); return 0; }\n')
    exe = str(tmp_path / "a")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-x",
                        "c", "-", "-o", exe], input=src, text=True, capture_output=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe], capture_output=True, text=True).stdout.split() == [
        str(N.SFFN_MX4), str(N.SFFN_MX4_MAX_K)]
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sparse_ffn_\w+)\s*\(", text)))
    assert set(names) == set(N.EXPORTED_MX4)
    out = subprocess.run(["nm", "-D", "--defined-only", N.LIB_PATH], capture_output=True,
                         text=True).stdout
    for name in names:
        assert re.search(rf"\bT {name}\b", out), name


def norm(N, **over):
    a = dict(x=A, dtype=1, ldx=100, res=A, ldr=100, rows=4, cols=100, w=A, wd=0, eps=1e-6, sum=A,
             ldsum=100, y=A, yd=4, ldy=64, scale=A, lds=16, stream=None)
    a.update(over)
    return N.lib().sparse_ffn_rms_norm(*a.values())


@pytest.mark.parametrize("over", [
    dict(x=None), dict(y=None), dict(scale=None), dict(dtype=3), dict(dtype=4), dict(dtype=-1),
    dict(yd=5), dict(yd=-1), dict(rows=-1), dict(cols=0), dict(ldx=99), dict(ldr=99), dict(ldsum=99),
    dict(res=None), dict(sum=None), dict(wd=3), dict(eps=-1e-6), dict(eps=math.inf), dict(eps=math.nan), dict(eps=1e-310),
    dict(ldy=48), dict(ldy=72), dict(lds=8), dict(lds=0), dict(lds=24), dict(y=A + 8), dict(scale=A + 4),
    dict(x=A + 1), dict(res=A + 1), dict(sum=A + 1), dict(w=A + 2),
    dict(yd=3, ldy=96), dict(yd=3, ldy=104), dict(yd=3, ldy=112, scale=None),
    dict(yd=3, ldy=112, scale=A + 2), dict(yd=3, ldy=112, y=A + 8),
    dict(yd=0, ldy=99, scale=None), dict(yd=0, ldy=100), dict(yd=0, ldy=100, scale=None, y=A + 2),
])
def test_norm_refuses(N, over):
    assert norm(N, **over) == N.SFFN_ERR_INVALID


def quantize(N, **over):
    a = dict(x=A, dtype=0, ldx=65, rows=4, cols=65, q=A, ldq=48, scale=A, lds=16, stream=None)
    a.update(over)
    return N.lib().sparse_ffn_quantize_mx4(*a.values())


@pytest.mark.parametrize("over", [
    dict(x=None), dict(q=None), dict(scale=None), dict(dtype=3), dict(dtype=4), dict(rows=-1),
    dict(cols=0), dict(ldx=64), dict(ldq=32), dict(ldq=56), dict(lds=3), dict(lds=20), dict(q=A + 8),
    dict(scale=A + 8), dict(x=A + 2),
])
def test_quantize_refuses(N, over):
    assert quantize(N, **over) == N.SFFN_ERR_INVALID


def dequantize(N, **over):
    a = dict(q=A, ldq=48, scale=A, lds=16, rows=4, cols=65, y=A, dtype=0, ldy=65, stream=None)
    a.update(over)
    return N.lib().sparse_ffn_dequantize_mx4(*a.values())


@pytest.mark.parametrize("over", [
    dict(q=None), dict(y=None), dict(scale=None), dict(dtype=3), dict(rows=-1), dict(cols=0),
    dict(ldy=64), dict(ldq=32), dict(ldq=56), dict(lds=2), dict(lds=20), dict(q=A + 8),
    dict(scale=A + 8), dict(y=A + 2),
])
def test_dequantize_refuses(N, over):
    assert dequantize(N, **over) == N.SFFN_ERR_INVALID


def matmul(lib, **over):
    a = dict(x=A, xd=1, xs=None, ldx=100, ldxs=0, M=5, K=100, w=A, ldw=64, ws=A, ldws=16, bias=None,
             N=7, y=A, yd=0, ldy=7, work=A, work_bytes=1 << 20, stream=None)
    a.update(over)
    return lib.lib().sparse_ffn_mx4_matmul(*a.values())


PACKED = dict(xd=4, xs=A, ldx=64, ldxs=16, K=128)
LONG = dict(M=50, K=600, ldx=600, ldw=304, ldws=32)  # x's rows are held in scratch


@pytest.mark.parametrize("over", [
    dict(x=None), dict(w=None), dict(ws=None), dict(y=None), dict(xd=3), dict(xd=5), dict(yd=3),
    dict(yd=4), dict(M=-1), dict(K=0), dict(N=0), dict(ldx=99), dict(ldy=6), dict(ldw=48),
    dict(ldw=72), dict(ldws=3), dict(ldws=20), dict(w=A + 8), dict(ws=A + 8), dict(x=A + 1),
    dict(y=A + 2), dict(xs=A), dict(bias=A + 2), dict(LONG, work=None), dict(LONG, work=A + 16),
    dict(LONG, work_bytes=16),
    dict(PACKED, xs=None), dict(PACKED, K=100), dict(PACKED, ldx=48), dict(PACKED, ldx=72),
    dict(PACKED, ldxs=2), dict(PACKED, ldxs=20), dict(PACKED, x=A + 8), dict(PACKED, xs=A + 8),
])
def test_matmul_refuses(N, over):
    assert matmul(N, **over) == N.SFFN_ERR_INVALID


def test_unsupported(N):
    K = N.SFFN_MX4_MAX_K + 1
    far = (1 << 24) + 16
    n = (1 << 31) - 1
    U = N.SFFN_ERR_UNSUPPORTED
    assert matmul(N, K=K, ldx=K, ldw=K + 15, ldws=K + 15) == U
    assert matmul(N, ldw=far) == U and matmul(N, ldws=far) == U
    assert matmul(N, **dict(PACKED, ldx=far)) == U and matmul(N, **dict(PACKED, ldxs=far)) == U
    assert matmul(N, M=n) == U and matmul(N, N=n, ldy=n) == U
    assert matmul(N, M=1 << 20, N=1 << 20, ldy=1 << 20) == U
    assert matmul(N, M=(1 << 31) - 1024) == U and matmul(N, M=(1 << 31) - 4096, x=None) == N.SFFN_ERR_INVALID
    assert quantize(N, cols=n, ldx=n, ldq=1 << 31, lds=1 << 27) == U
    assert quantize(N, ldq=far) == U and quantize(N, lds=far) == U
    assert dequantize(N, ldq=far) == U and dequantize(N, lds=far) == U
    assert norm(N, yd=0, scale=None, cols=n, ldx=n, ldr=n, ldsum=n, ldy=n) == U
    assert norm(N, ldy=far) == U
    wb = N.sparse_ffn_mx4_matmul_work_bytes
    none = C.c_size_t(-1).value
    for bad in ((0, 4, 4, K), (3, 4, 4, 64), (5, 4, 4, 64), (0, -1, 4, 64), (0, 4, 0, 64), (0, 4, 4, 0),
                (0, 1 << 31, 4, 64)):
        assert wb(*bad) == none, bad
    assert wb(0, 0, 4, 64) == 0
    # the product's own workgroups hold few rows, and short ones of few tiles; others lie in scratch
    assert wb(0, 4, 64, 20000) == wb(1, 50, 64, 512) == wb(2, 4096, 256, 1) == wb(4, 50, 64, 600) == 0
    assert wb(0, 50, 64, 513) > 0 and wb(0, 4097, 256, 64) > 0 and wb(0, 5, 64, 600) > 0
    with pytest.raises(N.SparseFFNError):
        N.sparse_ffn_quantize_mx4(A, 0, 1 << 33, 4, (1 << 32) + 32, A, 1 << 31, A, 1 << 27, None)


def test_no_rows_is_fine(N):
    assert norm(N, rows=0, x=None, y=None, scale=None, w=None) == N.SFFN_OK
    assert quantize(N, rows=0, x=None, q=None, scale=None) == N.SFFN_OK
    assert dequantize(N, rows=0, q=None, y=None, scale=None) == N.SFFN_OK
    assert matmul(N, M=0, x=None, w=None, ws=None, y=None, work=None, work_bytes=0) == N.SFFN_OK


def test_python_calls_want_device_tensors():
    import torch
    import activation_sparse_decode_rank_amd as P
    x = torch.zeros((2, 64))
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    for call in (lambda: P.rms_norm(x), lambda: P.quantize_mx4(x), lambda: P.dequantize_mx4(q, s),
                 lambda: P.mx4_matmul(x, q, s), lambda: P.rms_norm(x, out="i4"),
                 lambda: P.rms_norm(x.long()), lambda: P.mx4_matmul(q, q, s),
                 lambda: P.mx4_matmul(x, q, s, x_scale=s), lambda: P.dequantize_mx4(q, s, dtype=torch.int8),
                 lambda: P.rms_norm(x, residual_out=x)):
        with pytest.raises(ValueError):
            call()


def test_scratch_plan(tmp_path):
    """Codes and scales lie one behind the other, in whole groups of 16 blocks, each region from a
    multiple of 256 bytes on."""
    src = r'''
#include <cstdio>
#include <cstdlib>
#include <random>
#include "sffn_mx4_host.h"
using namespace sffn::host;
#define CHECK(c) do { if (!(c)) { std::printf("failed: %s line %d\n", #c, __LINE__); std::exit(1); } } while (0)
int main() {
  std::mt19937 g(7);
  for (int it = 0; it < 20000; ++it) {
    const int K = 1 + (int)(g() % (it % 3 ? 20000u : 1u << 20));
    const size_t M = 1 + g() % (it % 5 ? 5000u : 2147482624u);
    const int nb = mx4_blocks(K), np = mx4_padded(K);
    CHECK(nb * 32 >= K && (nb - 1) * 32 < K && np >= nb && np < nb + 16 && np % 16 == 0);
    const Mx4Carve c = mx4_carve(M, K);
    CHECK(c.q % 256 == 0 && c.scale % 256 == 0 && c.q + M * np * 16 <= c.scale);
    CHECK(c.scale + M * np <= c.bytes);
  }
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


def test_reference_holds_blocks_as_defined():
    """The plain form on values whose codes can be read off."""
    import numpy as np
    import mx4_ref as ref
    x = np.zeros((1, 40))
    x[0, :12] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6.9, -0.2, 0.26]
    x[0, 32:35] = [7, 3.5, 1.0]
    code, E = ref.blocks(x)
    assert E.tolist() == [[127, 128]]
    assert code[0, 0, :12].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 7, 8, 1]
    assert code[0, 1, :3].tolist() == [6, 4, 1]  # 3.5 -> 4, 1.75 -> 2, 0.5
    q, E = ref.pack(code, E)
    assert q[0, 0] == 0xF7 and ref.values(q, E)[0, :3].tolist() == [6, -6, 0]
    x[0, 3], x[0, 39] = np.nan, np.inf
    code, E = ref.blocks(x)
    assert E.tolist() == [[255, 255]] and not code.any()
    assert ref.blocks(np.full((1, 32), 2.0 ** -149))[1].tolist() == [[0]]


def test_calls_leave_what_is_not_regular():
    """The extension module takes device tensors only, and says so by None before it does anything."""
    import torch
    from activation_sparse_decode_rank_amd import _calls
    x = torch.zeros((2, 64))
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    assert _calls.norm(x, None, None, 1e-6, -1, None, 0, 0) is None
    assert _calls.norm([1.0], None, None, 1e-6, -1, None, 0, 0) is None
    assert _calls.quantize(x, 0, 0) is None and _calls.quantize("x", 0, 0) is None
    assert _calls.dequantize(q, s, -1, 0, 0, 0) is None
    assert _calls.matmul(x, q, s, None, None, -1, 0, 0) is None
    for call in (lambda: _calls.norm(x, None, None, "a", -1, None, 0, 0), lambda: _calls.bind(1),
                 lambda: _calls.quantize(x, "0", 0)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        _calls.bind(0, 0, 0, 0, 0)


def test_product_plan(tmp_path):
    """Every kernel is taken somewhere, at the sizes that the GPU test runs; a product in two launches
    covers every channel once, the first ones in whole tiles; launches stay within the device's limits
    for what the C call lets through."""
    import mx4_sizes
    names = {f: i for i, f in enumerate(("Few", "Short", "Split16", "Split16x32", "Split32", "Split64", "Tile64",
                                         "Tile64x128", "Tile128", "Tile256"))}
    want = "".join(f"  want({m}, {k}, {n}, kMx4{a}, {'kMx4' + b if b else -1});\n"
                   for a, b, m, k, n in mx4_sizes.FORMS)
    src = r'''
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include "sffn_mx4_host.h"
using namespace sffn::host;
#define CHECK(c) do { if (!(c)) { std::printf("failed: %s line %d\n", #c, __LINE__); std::exit(1); } } while (0)
static int seen[10];
static void want(size_t M, int K, size_t N, int form, int rest) {
  const Mx4Plan p = mx4_plan(M, N, mx4_blocks(K));
  if (p.form != form || (rest < 0 ? p.n1 != N : p.n1 >= N || p.rest != rest)) {
    std::printf("%zu x %d x %zu: form %d, rest %d from %zu on\n", M, K, N, p.form, p.rest, p.n1);
    std::exit(1);
  }
  seen[form]++;
}
int main() {
''' + want + r'''
  for (int f = 0; f < 10; ++f) CHECK(seen[f]);
  std::mt19937 g(11);
  auto pick = [&](double lo, double hi) { return (size_t)std::lround(std::exp(std::log(lo) + std::log(hi / lo) * (g() / 4294967296.0))); };
  for (int i = 0; i < 200000; ++i) {
    const size_t M = pick(1, i % 3 ? 1e4 : 2147482624.), N = pick(1, i % 2 ? 5e4 : 2147482624.);
    const int K = (int)pick(1, 1 << 20);
    if (!mx4_launches(M, N)) continue;  // refused
    const Mx4Plan p = mx4_plan(M, N, mx4_blocks(K));
    CHECK(p.n1 >= 1 && p.n1 <= N && (p.n1 == N || p.n1 % 256 == 0));
    auto one = [&](int form, size_t n) {
      static const size_t ch[] = {16, 16, 16, 16, 32, 64, 64, 64, 128, 256}, tk[] = {4, 16, 16, 32, 32, 64, 64, 128, 128, 256};
      static const size_t threads[] = {512, 512, 512, 512, 512, 512, 256, 256, 256, 512};
      CHECK(form != kMx4Few || (M <= 4 && mx4_few_lds(M, K) <= kMx4FewLds));
      CHECK((form == kMx4Short) == (M > 4 && mx4_blocks(K) <= 16 && (M + 15) / 16 * ((N + 15) / 16) <= kMx4ShortTiles));
      const size_t tiles = (n + ch[form] - 1) / ch[form] * ((M + tk[form] - 1) / tk[form]);
      if (form != kMx4Few) CHECK((tiles + 8) * threads[form] < (size_t)1 << 32);
    };
    one(p.form, p.n1);
    if (p.n1 < N) one(p.rest, N - p.n1);
  }
  std::puts("ok");
  return 0;
}
'''
    assert len(names) == 10
    (tmp_path / "plan.cpp").write_text(src)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I",
                    os.path.join(ROOT, "activation_sparse_decode_rank_amd", "csrc"),
                    str(tmp_path / "plan.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout
