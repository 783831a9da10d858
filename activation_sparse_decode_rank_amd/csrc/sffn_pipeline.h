// What the streaming and tiled products share: waits, loads straight into LDS, the exchange that
// turns whole lines into operands of the matrix cores, and how many workgroups a device holds.
#pragma once
#include <algorithm>
#include <atomic>

#include "sffn_device.h"

namespace sffn {
namespace {

typedef int int4_t __attribute__((ext_vector_type(4)));

// s_waitcnt operand (gfx9 encoding): LDS accesses only (lgkmcnt 0, vmcnt and expcnt at most)
constexpr int I8_WAIT_LGKM0 = 0xC07F;

// LDS accesses before it are done, in every wave of the workgroup, before any after it; loads
// from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(I8_WAIT_LGKM0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The stream of weights reads whole 128-byte lines: one load takes 8 rows x 128 bytes, lane
// (r16 = lane % 16, g = lane / 16) the 16-byte chunk g + 4 (r16 / 8) of row r16 % 8, and a second
// one the 8 rows after them. The matrix cores want chunk g (then 4 + g) of row r16 in that
// lane: the two loads' values change places between the halves of each 16 lanes. Loads of 16
// rows x 64 bytes need no change but halve the lines: 6.1 against 6.9 TB/s for a plain stream.
constexpr int DPP_ROW_ROR8 = 0x128;
__device__ __forceinline__ void to_steps(const int4_t& a, const int4_t& b, int4_t& s0, int4_t& s1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s0[i] = __builtin_amdgcn_update_dpp(a[i], b[i], DPP_ROW_ROR8, 0xF, 0xC, false);
    s1[i] = __builtin_amdgcn_update_dpp(b[i], a[i], DPP_ROW_ROR8, 0xF, 0x3, false);
  }
}

// this lane's 16 bytes at src to place 16 * lane of the 1 KB block at dst (LDS)
__device__ __forceinline__ void load_block(const int8_t* src, int8_t* dst) {
  __builtin_amdgcn_global_load_lds(reinterpret_cast<const u32x4*>(src),
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// until at most N of this wave's loads are in flight
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// instruction kinds of __builtin_amdgcn_sched_group_barrier
constexpr int SG_MFMA = 0x8, SG_LOAD = 0x20, SG_LDS_READ = 0x100;

// Workgroups of a kernel that the current device holds at once. The last answer is kept: device,
// dynamic LDS (below 2^24) and number in one word.
template <auto Kernel>
int resident(int threads, size_t lds) {
  static std::atomic<uint64_t> kept{0};
  int dev = 0, cus = 0, per = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 512;
  const uint64_t key = ((uint64_t)(dev + 1) << 48) | ((uint64_t)lds << 24);
  const uint64_t last = kept.load(std::memory_order_relaxed);
  if ((last & ~(uint64_t)0xFFFFFF) == key) return (int)(last & 0xFFFFFF);
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kernel, threads, lds) != hipSuccess)
    return 512;
  const int n = std::min(std::max(1, cus * per), 0xFFFFFF);
  kept.store(key | (uint64_t)n, std::memory_order_relaxed);
  return n;
}

}  // namespace
}  // namespace sffn
