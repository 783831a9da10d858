"""CPU tests of what the calls of include/sparse_ffn_experts.h refuse, or split up, at their
largest sizes: nothing is launched here."""
import ctypes as C
import os
import subprocess

import pytest

from test_experts_abi import A, N, desc, experts, matmul  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = (1 << 31) - 1


def test_channels_and_columns_near_32_bits_are_refused(N):  # noqa: F811
    """Tiles round channels, and rows of 16 bytes columns, up in 32 bits."""
    for n in (MOST, MOST - 100, MOST - 1022):
        assert matmul(N, N=n, ldy=n) == N.SFFN_ERR_UNSUPPORTED
        assert matmul(N, N=n, ldy=n, M=1, work=None, work_bytes=0) == N.SFFN_ERR_UNSUPPORTED
        a = dict(x=A, dtype=1, ldx=n, rows=1, cols=n, q=A, ldq=1 << 31, scale=A, stream=None)
        assert N.lib().sparse_ffn_quantize_rows(*a.values()) == N.SFFN_ERR_UNSUPPORTED


def test_products_past_one_launch_are_refused(N):  # noqa: F811
    """A launch holds less than 2^32 threads: 2^24 tiles of 64 rows x 128 channels are too many."""
    for M in (65, 96):
        assert matmul(N, M=M, N=1 << 30, ldy=1 << 30) == N.SFFN_ERR_UNSUPPORTED
    assert matmul(N, M=1 << 20, N=1 << 20, ldy=1 << 20) == N.SFFN_ERR_UNSUPPORTED


def build_and_run(tmp_path, body):
    """A C++ program over the host plan (csrc/sffn_i8_host.h), with its arithmetic checked."""
    src = r'''
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "sffn_i8_host.h"
using namespace sffn::host;
#define CHECK(c) do { if (!(c)) { std::printf("failed: %s line %d\n", #c, __LINE__); std::exit(1); } } while (0)
int main() {
''' + body + r'''
  std::puts("ok");
  return 0;
}
'''
    (tmp_path / "limits.cpp").write_text(src)
    exe = str(tmp_path / "limits")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "activation_sparse_decode_rank_amd", "csrc"),
                    str(tmp_path / "limits.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


def test_chunks_of_the_most_tokens(tmp_path):
    """The chunks of a call follow each other, without a gap, up to 2^31 - 1 tokens."""
    build_and_run(tmp_path, r'''
  for (int T : {1, 2, 1000, INT_MAX - 1, INT_MAX})
    for (int size : {1 << 24, (1 << 21) - 1, 12345678, 32768 / 3}) {
      if (T / size > 3000000) continue;
      const Chunks c(T, size);
      int64_t at = 0;
      for (int64_t i = 0; i < c.count; ++i) {
        CHECK(c.first(i) == at && c.tokens(i) >= 1 && c.tokens(i) <= size);
        at += c.tokens(i);
      }
      CHECK(at == T);
    }
''')


def test_launches_of_a_chunk_stay_below_32_bits_of_threads(tmp_path):
    """The rows into 8 bits (a workgroup of 1024 threads holds 16, 4 or 1 of them) and the sums
    over the slots (256 threads, four channels each), whatever scratch there is."""
    build_and_run(tmp_path, r'''
  for (int d : {1, 64, 1024, 1025, 4096, 4097, 16384, 70000, 131071})
    for (int k : {1, 2, 8, 64})
      for (int T : {1, 5000000, INT_MAX}) {
        const size_t c = experts_chunk(8, d, 64, T, k, (size_t)-1);
        CHECK(c >= 1 && c * k <= kExpertsMaxRows);
        const size_t rows = i8_kpad(d) <= 1024 ? 16 : i8_kpad(d) <= 4096 ? 4 : 1;
        CHECK((1 + (c + rows - 1) / rows) * 1024 < (size_t)1 << 32);
        CHECK(c * ((d + 1023) / 1024) * 256 < (size_t)1 << 32);
      }
''')


def test_order_of_chunks_by_trying_every_row(tmp_path):
    """Outputs over inputs: the order found is one that keeps the inputs, and one is found
    whenever there is one (forward first)."""
    build_and_run(tmp_path, r'''
  std::mt19937 g(11);
  auto pick = [&](int lo, int hi) { return lo + (int)(g() % (unsigned)(hi - lo + 1)); };
  int found[3] = {0, 0, 0};
  for (int it = 0; it < 200000; ++it) {
    const int T = pick(1, 40), size = pick(1, 12);
    const int xb = pick(1, 9), yb = pick(1, 9);
    const int xp = xb + pick(0, 9), yp = it % 3 ? yb + pick(0, 9) : std::max(xp, yb);
    const int64_t x = 1000 + pick(-200, 200), y = it % 5 ? 1000 + pick(-200, 200) : x;
    const Chunks c(T, size);
    bool later = false, earlier = false;
    for (int t = 0; t < T; ++t)
      for (int u = 0; u < T; ++u) {  // y's row t, x's row u
        const int64_t ya = y + (int64_t)t * yp, xa = x + (int64_t)u * xp;
        if (ya < xa + xb && xa < ya + yb) {
          later |= u / size > t / size;
          earlier |= u / size < t / size;
        }
      }
    const ChunkOrder want = !later ? ChunkOrder::Forward : !earlier ? ChunkOrder::Backward : ChunkOrder::None;
    CHECK(chunk_order(c, x, xp, xb, y, yp, yb) == want);
    if (x == y) CHECK(want != ChunkOrder::None);
    found[(int)want]++;
  }
  CHECK(found[0] > 1000 && found[1] > 1000 && found[2] > 1000);
  const Chunks most(INT_MAX, 7);  // rows as far apart as 64 bits hold
  CHECK(chunk_order(most, 4096, LLONG_MAX, 64, 4096, LLONG_MAX, 64) == ChunkOrder::Forward);
''')


BIG = 1 << 32


@pytest.mark.parametrize("name,args,at", [
    ("route", [A, 1, 64, 4, 64, 8, 0, None, 1, 1, 1, 1, 1.0, A, A, None], (3, 4, 5, 6, 8, 9, 10)),
    ("quantize_rows", [A, 1, 32, 4, 32, A, 32, A, None], (3, 4)),
    ("i8_matmul", [A, 1, None, 64, 3, 64, A, 64, A, None, 16, A, 0, 16, None, 0, None], (4, 5, 10)),
    ("experts", [None, A, 1, 64, 3, A, A, 2, A, 1, 64, A, 1 << 24, None], (4, 7)),
])
def test_python_does_not_cut_integers_to_32_bits(N, name, args, at):  # noqa: F811
    """Numbers that fit the call's 32 bits only when cut to them are refused, not cut."""
    call = getattr(N, "sparse_ffn_" + name)
    if name == "experts":
        args[0] = desc(N)
    for i in at:
        for v, status in ((args[i] + BIG, N.SFFN_ERR_UNSUPPORTED), (args[i] - BIG, N.SFFN_ERR_INVALID)):
            wrong = list(args)
            wrong[i] = v
            with pytest.raises(N.SparseFFNError) as e:
                call(*wrong)
            assert e.value.status == status, (i, v)


def test_size_queries_do_not_cut_integers_to_32_bits(N):  # noqa: F811
    none = C.c_size_t(-1).value
    for sizes in ((4 + BIG, 16, 64), (4, 16 + BIG, 64), (4, 16, 64 + BIG), (4 - BIG, 16, 64)):
        assert N.sparse_ffn_i8_matmul_work_bytes(3, *sizes) == none
    wb = N.sparse_ffn_experts_work_bytes
    assert wb(desc(N), 4 + BIG, 2) == wb(desc(N), 4, 2 + BIG) == wb(desc(N), 4 - BIG, 2) == 0


def test_shapes_past_32_bits_are_refused():
    import torch
    import activation_sparse_decode_rank_amd as P
    many = torch.empty((5, 1), dtype=torch.int8).as_strided((1, BIG + 2, 1), (0, 0, 1))
    one = torch.ones((1, 1))
    with pytest.raises(ValueError, match="32 bits"):
        P.experts(one, one.int(), one, many, one, many, one)
