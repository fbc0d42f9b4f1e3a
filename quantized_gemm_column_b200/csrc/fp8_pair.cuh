// What the 8-bit products on CTA pairs share: single-thread roles, TMA loads
// and MMAs, and the experts' buffer from the counts.
#pragma once

#include "device.cuh"
#include "pair.cuh"
#include "route.h"

namespace avr {
namespace fp8 {

// TMA 2-D load into this CTA's shared memory, completing on the barrier at a
// shared::cluster address in either CTA of the pair
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t x,
                                                 int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}

// One lane of a converged warp.  The compiler knows that the branch on it has
// one thread, which a branch on the lane number does not tell it: issued from
// the latter, the MMAs, commits and copies of a stage took about 290 ns more
// (8192 x 1024 x 4096: 36.8 -> 27.6 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void mma_fp8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t"
      "}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// The experts' buffer in shared memory
struct Buffer {
  int32_t rows[kMaxExperts];       // tokens
  int32_t blk_end[kMaxExperts];    // 128-row blocks up to and with this expert
  int32_t tile_end[kMaxExperts];   // row tiles likewise
  uint64_t warp[32];
};

// Fills it from the counts, by the whole CTA; the number of row tiles (of
// kBlocks 128-row blocks of one expert), 0 when the segments do not fit l_cap rows.
template <int kThreads, int kBlocks>
__device__ __forceinline__ int scan_counts(const int32_t* counts, int E, int64_t l_cap, Buffer* b, uint32_t* status) {
  static_assert(2 * kThreads >= kMaxExperts, "two experts a thread");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t n[2];
  uint64_t x[2];
  bool bad = false;
  // blocks in the low 35 bits of a word (1024 counts of at most 2^24 blocks),
  // tiles above them: when the segments fit there are at most 2^24 tiles
  constexpr int kShift = 35;
  constexpr uint64_t kLow = (1ull << kShift) - 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    n[i] = 2 * tid + i < E ? __ldcg(counts + 2 * tid + i) : 0;
    const bool out = n[i] < 0 || n[i] > l_cap;
    bad |= out;
    const uint64_t blk = out ? 0 : (static_cast<uint64_t>(n[i]) + 127) / 128;
    x[i] = blk | (((blk + kBlocks - 1) / kBlocks) << kShift);
  }
  uint64_t sum = x[0] + x[1];
  const uint64_t own = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) b->warp[warp] = sum;
  const bool any_bad = __syncthreads_or(bad) != 0;
  uint64_t before = sum - own, all = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    before += w < warp ? b->warp[w] : 0;
    all += b->warp[w];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    before += x[i];
    if (2 * tid + i < E) {
      b->rows[2 * tid + i] = n[i];
      b->blk_end[2 * tid + i] = static_cast<int32_t>(before & kLow);
      b->tile_end[2 * tid + i] = static_cast<int32_t>(before >> kShift);
    }
  }
  const bool fits = !any_bad && static_cast<int64_t>(all & kLow) <= l_cap / 128;
  if (!fits && blockIdx.x == 0 && tid == 0) raise_status(status, AVR_ERR_INVALID_ARG);
  __syncthreads();
  return fits ? static_cast<int>(all >> kShift) : 0;
}

// the expert of row tile mt
__device__ __forceinline__ int expert_of_tile(const Buffer* b, int E, int mt) {
  int lo = 0, hi = E - 1;                  // the first whose tiles end past mt
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (b->tile_end[mid] > mt)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

}  // namespace fp8
}  // namespace avr
