// Routing of a mixture of experts: the router and its gradient, the sort of
// tokens by expert, dispatch to the experts' buffer and combine with their
// gradients (the formulas are in include/averis.h).
//
// None of these kernels has arithmetic to speak of: the router and the sort
// of a decoding step are bound by launch latency, the rest by the bytes of
// the buffers, each moved once.
#include <cuda_bf16.h>

#include "device.cuh"
#include "route.h"
#include "strips.cuh"

namespace avr {

namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

template <bool kBf16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}
template <bool kBf16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (kBf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

// 16 bytes of the tensors' type as fp32 values and back
template <bool kBf16>
struct Vec {
  static constexpr int kN = kBf16 ? 8 : 4;
};
template <bool kBf16>
__device__ __forceinline__ void unpack(const uint4& q, float (&f)[Vec<kBf16>::kN]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kBf16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}
template <bool kBf16>
__device__ __forceinline__ uint4 pack(const float (&f)[Vec<kBf16>::kN]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kBf16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      w[i] = __float_as_uint(f[i]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// the values of one 16-byte vector (of kBf16) to vector i of a tensor of kBf16Out
template <bool kBf16, bool kBf16Out>
__device__ __forceinline__ void store_vec(void* dst, int64_t i, const float (&f)[Vec<kBf16>::kN]) {
  if constexpr (kBf16 == kBf16Out) {
    static_cast<uint4*>(dst)[i] = pack<kBf16>(f);
  } else {
    static_assert(!kBf16, "fp32 to bf16");
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    static_cast<uint2*>(dst)[i] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// router: one warp per token, experts NV lane .. NV lane + NV - 1 in a lane's
// registers, so that a lower lane holds lower experts
// ---------------------------------------------------------------------------
// Warps of a block.  A GPU starts about one block in a nanosecond, which with
// 4 warps is all the time that many tokens of few experts take: the gradient
// of 32768 tokens of 128 experts with `norm` takes 5.2 us with 8 and 8.9 with
// 4 (12: 5.1), the router's 16 experts 7.7 and 9.0.  Beyond 128 experts a
// token works longer and larger blocks end unevenly: 4096 tokens of 256
// experts 5.4 with 8, 5.0 with 4.
__host__ __device__ constexpr int route_warps(int nv) { return nv <= 4 ? 8 : 4; }

// the NV values of a lane from e0 on, -inf past E; wide: rows can be read and
// written min(NV, 4) values at a time
template <bool kBf16, int NV>
__device__ __forceinline__ void load_lane(const void* row, int e0, int E, bool wide, float (&v)[NV]) {
  constexpr int W = NV < 4 ? NV : 4;
  if (wide && W > 1) {
#pragma unroll
    for (int i = 0; i < NV; i += W) {
      uint32_t w[4] = {};
      const bool in = e0 + i < E;
      if (kBf16) {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(row) + e0 + i;
        if (in && W == 4) {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          w[0] = x.x << 16, w[1] = x.x & 0xFFFF0000u, w[2] = x.y << 16, w[3] = x.y & 0xFFFF0000u;
        } else if (in) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
          w[0] = x << 16, w[1] = x & 0xFFFF0000u;
        }
      } else {
        const float* p = static_cast<const float*>(row) + e0 + i;
        if (in && W == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(p);
          w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else if (in) {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          w[0] = x.x, w[1] = x.y;
        }
      }
#pragma unroll
      for (int c = 0; c < W; ++c) v[i + c] = in ? __uint_as_float(w[c]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = e0 + i < E ? load1<kBf16>(row, e0 + i) : -INFINITY;
  }
}
template <bool kBf16, int NV>
__device__ __forceinline__ void store_lane(void* row, int e0, int E, bool wide, const float (&v)[NV]) {
  constexpr int W = NV < 4 ? NV : 4;
  if (wide && W > 1) {
#pragma unroll
    for (int i = 0; i < NV; i += W) {
      if (e0 + i >= E) continue;
      if (kBf16) {
        uint32_t w[W / 2 > 0 ? W / 2 : 1];
#pragma unroll
        for (int c = 0; c < W / 2; ++c) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[i + 2 * c], v[i + 2 * c + 1]);
          w[c] = *reinterpret_cast<const uint32_t*>(&x);
        }
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(row) + e0 + i;
        if (W == 4)
          *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[W / 2 - 1]);
        else
          *reinterpret_cast<uint32_t*>(p) = w[0];
      } else {
        float* p = static_cast<float*>(row) + e0 + i;
        if (W == 4)
          *reinterpret_cast<float4*>(p) = make_float4(v[i], v[i + 1], v[i + W - 2], v[i + W - 1]);
        else
          *reinterpret_cast<float2*>(p) = make_float2(v[i], v[i + W - 1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < E) store1<kBf16>(row, e0 + i, v[i]);
  }
}
template <bool kBf16>
__device__ __forceinline__ const void* row_of(const void* p, int64_t at) {
  return kBf16 ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(p) + at)
               : static_cast<const void*>(static_cast<const float*>(p) + at);
}

// a key that orders as the value does, above 0 for every value but -inf (and
// NaN); + 0.0f makes the two zeros one value
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t u = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return v > -INFINITY ? u : 0u;
}

__device__ __forceinline__ float key_value(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Each of the k steps takes the largest key of the warp and, among the lanes
// that hold it, the lowest expert.  What bounds this is the number of
// instructions, 423 a token of 128 experts with 8 slots, of which 39 % go to
// the pipe of half rate (the schedulers issue in 82 % of their cycles, that
// pipe is busy in 64 %, and the logits are 17 MB for 32768 tokens), so a
// step is kept short: a lane sorts its keys once (descending, the lower expert
// first among equal ones; for up to 8, beyond that it searches), its best is
// always the first, and the lowest lane that holds the step's maximum notes its
// expert in shared memory and moves up by one.  A lane's experts are
// neighbours, so its row comes in one wide load and ties need no second
// reduction: 32768 tokens of 128 experts, 8 slots, take 14.9 us (13.9 with
// `norm`), with experts 32 apart and a vote on ties 16.7 (15.7); 256 experts
// 27.0 against 29.6.  The gradient of the 128 experts' tokens takes 9.5 us (5.4
// with `norm`, which reads no logits).  From 257 experts on, a step searches the
// lane's 16 or 32 keys: 32768 tokens of 512 experts take 45 us with 8 slots and
// 134 with 32, of 1024 experts 80 and 239 (their logits are read in 10 and 20).
template <bool kBf16, int NV>
__global__ void __launch_bounds__(32 * route_warps(NV))
    route_kernel(const void* logits, int64_t T, int E, int k, int norm, bool wide, int32_t* ids, float* weights,
                 uint32_t* status) {
  __shared__ int32_t s_slot[route_warps(NV)][kMaxSlots];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int lane = threadIdx.x & 31;
  int32_t* slot = s_slot[threadIdx.x >> 5];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * route_warps(NV) + (threadIdx.x >> 5);
  if (t >= T) return;
  const int e0 = NV * lane;
  float v[NV];
  uint32_t key[NV];
  bool bad = false;
  load_lane<kBf16, NV>(row_of<kBf16>(logits, t * E), e0, E, wide, v);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    bad |= !(v[i] < INFINITY);
    key[i] = order_key(v[i]);
  }
  if (__any_sync(kFull, bad)) {       // NaN or +inf: the token goes without experts
    if (lane == 0) raise_status(status, AVR_ERR_NONFINITE);
    if (lane < k) {
      ids[t * k + lane] = -1;
      weights[t * k + lane] = 0.0f;
    }
    return;
  }
  constexpr bool kSort = NV <= 8;
  uint32_t order = 0x76543210u;       // kSort: which of the lane's experts the keys are, four bits each
  if (kSort) {
    // odd-even transposition: neighbours swap only when strictly out of order, so equal keys keep theirs
    uint32_t at[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) at[i] = i;
#pragma unroll
    for (int r = 0; r < NV; ++r) {
#pragma unroll
      for (int i = r & 1; i + 1 < NV; i += 2) {
        const bool swap = key[i] < key[i + 1];
        const uint32_t x = swap ? key[i + 1] : key[i], y = swap ? key[i] : key[i + 1];
        const uint32_t ax = swap ? at[i + 1] : at[i], ay = swap ? at[i] : at[i + 1];
        key[i] = x;
        key[i + 1] = y;
        at[i] = ax;
        at[i + 1] = ay;
      }
    }
    order = at[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) order |= at[i] << (4 * i);
  }
  uint32_t my_key = 0u;               // lane j holds slot j
  int taken = 0;
  for (; taken < k; ++taken) {
    uint32_t best = key[0];
    uint32_t best_at = kSort ? order & 15u : 0u;
    if (!kSort) {
#pragma unroll
      for (int i = 1; i < NV; ++i) {
        if (key[i] > best) {          // strictly: the lower expert of equal ones
          best = key[i];
          best_at = i;
        }
      }
    }
    const uint32_t m = __reduce_max_sync(kFull, best);
    if (m == 0u) break;               // only -inf left
    const bool mine = __ffs(__ballot_sync(kFull, best == m)) == lane + 1;
    if (lane == taken) my_key = m;
    if (mine) {
      slot[taken] = e0 + static_cast<int32_t>(best_at);
      if (kSort) {
        order >>= 4;
#pragma unroll
        for (int i = 0; i + 1 < NV; ++i) key[i] = key[i + 1];
        key[NV - 1] = 0u;
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i == static_cast<int>(best_at)) key[i] = 0u;
      }
    }
  }
  __syncwarp();
  const float top = key_value(__shfl_sync(kFull, my_key, 0));
  const float mine = lane < taken ? expf(key_value(my_key) - top) : 0.0f;
  float den = mine;
  if (!norm && taken > 0) {
    den = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) den += expf(v[i] - top);
  }
  den = warp_sum(den);
  if (lane < k) {
    ids[t * k + lane] = lane < taken ? slot[lane] : -1;
    weights[t * k + lane] = lane < taken ? mine / den : 0.0f;
  }
}

// Gradient: lane j holds slot j; the chosen experts' terms are added into a
// row of shared memory, so the logits' loop needs no search.
template <bool kBf16, int NV>
__global__ void __launch_bounds__(32 * route_warps(NV))
    route_bwd_kernel(const void* logits, int64_t T, int E, int k, int norm, bool wide, const int32_t* ids,
                     const float* weights, const float* dweights, void* dlogits, uint32_t* status) {
  __shared__ __align__(16) float s_row[route_warps(NV)][32 * NV];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int lane = threadIdx.x & 31;
  float* row = s_row[threadIdx.x >> 5];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * route_warps(NV) + (threadIdx.x >> 5);
  if (t >= T) return;
  const int e0 = NV * lane;
  float v[NV];
  if (!norm) load_lane<kBf16, NV>(row_of<kBf16>(logits, t * E), e0, E, wide, v);
  int id = -1;
  float w = 0.0f, dw = 0.0f;
  if (lane < k) {                     // the three loads in flight together; an empty slot's values are not used
    id = ids[t * k + lane];
    w = weights[t * k + lane];
    dw = dweights[t * k + lane];
    if (id >= E) {
      raise_status(status, AVR_ERR_INVALID_ARG);
      id = -1;
    }
    if (id < 0) w = dw = 0.0f;
  }
  float s = w * dw, den = 0.0f;
  if (!norm) {
    uint32_t top_key = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) top_key = max(top_key, order_key(v[i]));
    top_key = __reduce_max_sync(kFull, top_key);
    const float top = key_value(top_key);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = top_key != 0u ? expf(v[i] - top) : 0.0f;       // 0: every logit is -inf
      den += v[i];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {  // both sums, one chain of shuffles
    s += __shfl_xor_sync(kFull, s, o);
    den += __shfl_xor_sync(kFull, den, o);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) row[e0 + i] = 0.0f;
  __syncwarp();
  // every slot leaves its number at its expert; a slot that finds another's
  // there shares the expert with it (a row that names one twice)
  const float g = norm ? w * (dw - s) : w * dw;
  if (id >= 0) row[id] = __int_as_float(lane);
  __syncwarp();
  const bool shared = id >= 0 && __float_as_int(row[id]) != lane;
  const bool any_shared = __any_sync(kFull, shared);
  if (id >= 0) row[id] = any_shared ? 0.0f : g;
  __syncwarp();
  if (any_shared) {                   // then one slot after another
    for (int j = 0; j < k; ++j) {
      if (lane == j && id >= 0) row[id] += g;
      __syncwarp();
    }
  }
  float d[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) d[i] = row[e0 + i];
  void* out = const_cast<void*>(row_of<kBf16>(dlogits, t * E));
  // a token without experts (a NaN or +inf logit leaves it so) has gradient 0,
  // whatever its logits' exponentials are
  if (norm || !__any_sync(kFull, id >= 0)) {
    store_lane<kBf16, NV>(out, e0, E, wide, d);
    return;
  }
  const float c = den == 0.0f ? 0.0f : s / den;        // 0: every logit is -inf
#pragma unroll
  for (int i = 0; i < NV; ++i) d[i] -= v[i] * c;
  store_lane<kBf16, NV>(out, e0, E, wide, d);
}

template <bool kBf16, int NV>
static cudaError_t route_t(const void* logits, int64_t T, int E, int k, int norm, int32_t* ids, float* weights,
                           const float* dweights, void* dlogits, uint32_t* status, cudaStream_t s) {
  constexpr int kWarps = route_warps(NV);
  const dim3 grid(static_cast<unsigned>((T + kWarps - 1) / kWarps));
  const bool wide = E % (NV < 4 ? NV : 4) == 0;        // the tensors start on 16 bytes
  if (dlogits == nullptr)
    return launch_ex(route_kernel<kBf16, NV>, grid, dim3(32 * kWarps), 0, s, true, logits, T, E, k, norm,
                     wide, ids, weights, status);
  return launch_ex(route_bwd_kernel<kBf16, NV>, grid, dim3(32 * kWarps), 0, s, true, logits, T, E, k, norm,
                   wide, ids, weights, dweights, dlogits, status);
}

template <bool kBf16>
static cudaError_t route_d(const void* logits, int64_t T, int E, int k, int norm, int32_t* ids, float* weights,
                           const float* dweights, void* dlogits, uint32_t* status, cudaStream_t s) {
#define AVR_ROUTE(NV) \
  if (E <= 32 * NV) return route_t<kBf16, NV>(logits, T, E, k, norm, ids, weights, dweights, dlogits, status, s)
  AVR_ROUTE(1);
  AVR_ROUTE(2);
  AVR_ROUTE(4);
  AVR_ROUTE(8);
  AVR_ROUTE(16);
  AVR_ROUTE(32);
#undef AVR_ROUTE
  return cudaErrorInvalidValue;
}

cudaError_t launch_route(const void* logits, avr_dtype lt, int64_t T, int E, int k, int norm, int32_t* ids,
                         float* weights, uint32_t* status, cudaStream_t s) {
  return lt == AVR_BF16 ? route_d<true>(logits, T, E, k, norm, ids, weights, nullptr, nullptr, status, s)
                        : route_d<false>(logits, T, E, k, norm, ids, weights, nullptr, nullptr, status, s);
}

cudaError_t launch_route_bwd(const void* logits, avr_dtype lt, int64_t T, int E, int k, int norm, const int32_t* ids,
                             const float* weights, const float* dweights, void* dlogits, uint32_t* status,
                             cudaStream_t s) {
  int32_t* i = const_cast<int32_t*>(ids);
  float* w = const_cast<float*>(weights);
  return lt == AVR_BF16 ? route_d<true>(logits, T, E, k, norm, i, w, dweights, dlogits, status, s)
                        : route_d<false>(logits, T, E, k, norm, i, w, dweights, dlogits, status, s);
}

// ---------------------------------------------------------------------------
// sort by expert: a stable counting sort over G chunks of consecutive slots.
// Kernel 1 counts each chunk's slots per expert; in kernel 2 every CTA adds up
// the counts of the chunks before its own (a few tens of KB from L2), scans
// the padded totals over the experts, and ranks its slots.  One chunk needs
// only kernel 2, which then counts its slots itself.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
// A decoding step's slots take one round of one smaller block, whose barriers
// and cleared counts are cheaper.  us with 256 threads / with 1024, 64 experts:
// 64 slots 2.1 / 2.9, 256 slots 2.3 / 3.0, 384 slots 2.9 / 3.0, 512 slots 3.3 /
// 3.3, 1024 slots 4.7 / 3.8.  A thread is an expert in the scan, so E is bounded
// too.
constexpr int kFewSlots = 256;
static_assert(kSortThreads >= kMaxExperts, "one thread an expert");

int sort_chunks(int64_t slots) {
  const int64_t g = (slots + kSortThreads - 1) / kSortThreads;
  return static_cast<int>(g < 1 ? 1 : g > 128 ? 128 : g);
}

// expert of slot i, -1 for none (and for an id that no expert has)
__device__ __forceinline__ int slot_expert(const int32_t* ids, int64_t i, int64_t end, int E, bool& bad) {
  const int e = i < end ? __ldg(ids + i) : -1;
  bad |= e >= E;
  return e >= E ? -1 : e;
}

template <int kT>
__device__ __forceinline__ void count_chunk(const int32_t* ids, int64_t lo, int64_t hi, int E, int32_t* s_cnt,
                                            uint32_t* status) {
  bool bad = false;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kT) {
    const int e = slot_expert(ids, i, hi, E, bad);
    if (e >= 0) atomicAdd(&s_cnt[e], 1);      // integers: any order gives the same counts
  }
  if (bad) raise_status(status, AVR_ERR_INVALID_ARG);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int32_t* ids, int64_t slots, int64_t per,
                                                                  int E, int32_t* hist, uint32_t* status) {
  __shared__ int32_t s_cnt[kMaxExperts];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  for (int e = threadIdx.x; e < E; e += kSortThreads) s_cnt[e] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * per;
  count_chunk<kSortThreads>(ids, lo, min64(slots, lo + per), E, s_cnt, status);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[static_cast<int64_t>(blockIdx.x) * E + e] = s_cnt[e];
}

template <int kT>
__global__ void __launch_bounds__(kT)
    sort_place_kernel(const int32_t* ids, int64_t slots, int64_t per, int E, int64_t l_cap, const int32_t* hist,
                      int32_t* counts, int32_t* row, uint32_t* status) {
  constexpr int kWarps = kT / 32;
  __shared__ int32_t s_total[kT];    // all slots of an expert
  __shared__ int32_t s_next[kT];     // the buffer row of this chunk's next slot of an expert
  __shared__ int64_t s_warp[kWarps];
  extern __shared__ uint16_t s_in[];          // [kWarps][E] slots of a round, per warp
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int G = static_cast<int>(gridDim.x), g = static_cast<int>(blockIdx.x);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t lo = g * per, hi = min64(slots, lo + per);
  for (int e = tid; e < E; e += kT) {
    s_total[e] = 0;
    s_next[e] = 0;
  }
  __syncthreads();
  if (G == 1) {
    count_chunk<kT>(ids, lo, hi, E, s_total, status);
  } else {
    // thread (slice, e): the chunks slice, slice + slices, ... of expert e
    int ep = 32;
    while (ep < E) ep <<= 1;
    const int e = tid & (ep - 1), slices = kT / ep;
    if (e < E) {
      int32_t all = 0, before = 0;
      for (int c = tid / ep; c < G; c += slices) {
        const int32_t n = __ldcg(hist + static_cast<int64_t>(c) * E + e);
        all += n;
        before += c < g ? n : 0;
      }
      atomicAdd(&s_total[e], all);
      atomicAdd(&s_next[e], before);
    }
  }
  __syncthreads();
  // exclusive scan of the padded totals over the experts (thread = expert)
  const int64_t n = tid < E ? s_total[tid] : 0;
  const int64_t pad = (n + 127) / 128 * 128;
  int64_t x = pad;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t y = lane < kWarps ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(kFull, y, o);
      if (lane >= o) y += z;
    }
    if (lane < kWarps) s_warp[lane] = y;
  }
  __syncthreads();
  const int64_t first = x - pad + (warp > 0 ? s_warp[warp - 1] : 0);
  const bool fits = s_warp[kWarps - 1] <= l_cap;
  if (tid < E) {
    s_next[tid] += static_cast<int32_t>(first);     // fits: below 2^31; unused otherwise
    if (g == 0) counts[tid] = fits ? static_cast<int32_t>(n) : 0;
  }
  if (!fits) {
    if (g == 0 && tid == 0) raise_status(status, AVR_ERR_INVALID_ARG);
    for (int64_t i = lo + tid; i < hi; i += kT) row[i] = -1;
    return;
  }
  // rounds of kT consecutive slots: rank inside the warp, then the warps in order
  uint16_t* mine = s_in + warp * E;
  for (int64_t base = lo; base < hi; base += kT) {
    for (int i = tid; i < kWarps * E; i += kT) s_in[i] = 0;
    __syncthreads();
    bool bad = false;
    const int64_t i = base + tid;
    const int e = slot_expert(ids, i, hi, E, bad);
    const uint32_t same = __match_any_sync(kFull, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) mine[e] = static_cast<uint16_t>(__popc(same));
    __syncthreads();
    if (tid < E) {
      int32_t at = 0;
#pragma unroll 8
      for (int w = 0; w < kWarps; ++w) {
        const int32_t c = s_in[w * E + tid];
        s_in[w * E + tid] = static_cast<uint16_t>(at);
        at += c;
      }
      s_total[tid] = at;                      // this round's slots of the expert
    }
    __syncthreads();
    if (i < hi) row[i] = e >= 0 ? s_next[e] + mine[e] + rank : -1;
    __syncthreads();
    if (tid < E) s_next[tid] += s_total[tid];
  }
}

template <int kT>
static cudaError_t place_t(const int32_t* ids, int64_t slots, int64_t per, int G, int E, int64_t l_cap,
                           int32_t* counts, int32_t* row, const int32_t* scratch, uint32_t* status, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kT / 32) * static_cast<size_t>(E) * sizeof(uint16_t);
  auto kern = sort_place_kernel<kT>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_ex(kern, dim3(G), dim3(kT), smem, s, true, ids, slots, per, E, l_cap, scratch, counts, row, status);
}

cudaError_t launch_sort(const int32_t* ids, int64_t slots, int E, int64_t l_cap, int32_t* counts, int32_t* row,
                        int32_t* scratch, uint32_t* status, cudaStream_t s) {
  const int G = sort_chunks(slots);
  const int64_t per = (slots + G - 1) / G;
  if (slots <= kFewSlots && E <= kFewSlots)
    return place_t<kFewSlots>(ids, slots, per, G, E, l_cap, counts, row, scratch, status, s);
  if (G > 1) {
    cudaError_t e = launch_ex(sort_count_kernel, dim3(G), dim3(kSortThreads), 0, s, true, ids, slots, per, E, scratch,
                              status);
    if (e != cudaSuccess) return e;
  }
  return place_t<kSortThreads>(ids, slots, per, G, E, l_cap, counts, row, scratch, status, s);
}

// ---------------------------------------------------------------------------
// dispatch, combine and their gradients.  All go token by token: a token's
// row of X, Y or dY is moved once whatever k is, and the buffer's rows once
// each.  A warp takes (token, strip of 32 lanes x kU 16-byte vectors).
// ---------------------------------------------------------------------------
constexpr int kPermThreads = 128;

// the buffer row of slot (t, j), -1 for none
__device__ __forceinline__ int64_t slot_row(const PermuteArgs& a, int64_t t, int j) {
  const int32_t r = __ldg(a.row + t * a.k + j);
  if (r >= a.l_cap) {
    raise_status(a.status, AVR_ERR_INVALID_ARG);
    return -1;
  }
  return r;
}

// With few tokens (T times the 16-byte vectors of a row up to this) a strip is
// one vector a lane, so that the work spreads over four times the warps and
// all of a token's loads are in flight together.  us with one vector a lane /
// with four, 2048 bf16, 8 slots (thousands of vectors):
//   tokens (vectors)   64 (16)      128 (33)     256 (66)     512 (131)
//   dispatch           1.8 / 2.3    1.9 / 2.4    2.6 / 2.6    3.8 / 3.7
//   combine            3.2 / 3.5    3.3 / 3.5    3.5 / 3.6    5.3 / 4.2
// An fp32 buffer into bf16 tokens is even later with 8 slots (256 tokens of
// 2048, 131 thousand vectors: 3.5 / 4.4) and earlier with 2 (512 tokens of 1024,
// as many vectors: 2.2 / 2.0).
constexpr int64_t kFewVectors = 32768;

template <int kU>
__global__ void __launch_bounds__(kPermThreads) dispatch_kernel(const PermuteArgs a, int64_t V, int strips) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kPermThreads / 32);
  const uint4* src = static_cast<const uint4*>(a.src);
  uint4* dst = static_cast<uint4*>(a.dst);
  for (StripWalk at(static_cast<int64_t>(blockIdx.x) * (kPermThreads / 32) + (threadIdx.x >> 5), warps, a.T * strips,
                    strips);
       at.more(); at.step()) {
    const int64_t t = at.row;
    const int64_t v0 = static_cast<int64_t>(at.strip) * (32 * kU) + lane;
    // many tokens: the cached index costs less than the lanes' exchange (48.5 us against 49.8)
    const int row = kU == 1 && lane < a.k ? static_cast<int>(slot_row(a, t, lane)) : -1;
    uint4 q[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (v0 + 32 * u < V) q[u] = __ldg(src + t * V + v0 + 32 * u);
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = kU == 1 ? __shfl_sync(kFull, row, j) : slot_row(a, t, j);
      if (r < 0) continue;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (v0 + 32 * u < V) dst[r * V + v0 + 32 * u] = q[u];
    }
  }
}

// With many tokens a strip is 2 KB of each of the token's rows.  Longer pieces of a row at a
// time are what HBM wants: 512-byte strips with more slots' loads in flight
// took 66-73 us where these take 52 (8192 tokens, 8 slots, 2048 bf16).  The
// token's rows and weights are held by lanes, so that no load of a vector
// waits for one of an index.  kBf16 is the buffer's type, kBf16Out the tokens':
// an fp32 buffer (twice the bytes) takes 85 us for the same tokens (6.6 TB/s).
template <bool kBf16, bool kBf16Out, bool kWeighted, int kU>
__global__ void __launch_bounds__(kPermThreads, 4) combine_kernel(const PermuteArgs a, int64_t V, int strips) {
  constexpr int N = Vec<kBf16>::kN;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kPermThreads / 32);
  const uint4* src = static_cast<const uint4*>(a.src);
  for (StripWalk at(static_cast<int64_t>(blockIdx.x) * (kPermThreads / 32) + (threadIdx.x >> 5), warps, a.T * strips,
                    strips);
       at.more(); at.step()) {
    const int64_t t = at.row;
    const int64_t v0 = static_cast<int64_t>(at.strip) * (32 * kU) + lane;
    const int row = lane < a.k ? static_cast<int>(slot_row(a, t, lane)) : -1;
    const float weight = kWeighted && row >= 0 ? __ldg(a.weights + t * a.k + lane) : 0.0f;
    float acc[kU][N] = {};
#pragma unroll(kU == 1 ? 8 : 2)
    for (int j = 0; j < a.k; ++j) {
      const int r = __shfl_sync(kFull, row, j);
      const float w = __shfl_sync(kFull, weight, j);
      if (r < 0) continue;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (v0 + 32 * u < V) {
          float f[N];
          unpack<kBf16>(__ldg(src + r * V + v0 + 32 * u), f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[u][i] = kWeighted ? fmaf(w, f[i], acc[u][i]) : acc[u][i] + f[i];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (v0 + 32 * u < V) store_vec<kBf16, kBf16Out>(a.dst, t * V + v0 + 32 * u, acc[u]);
  }
}

// One CTA per token: dY's row stays in L1 over the slots, and the dot products
// of all slots are summed in the same order whatever the grid.  The block has
// as many threads as make whole passes over the row's vectors, 128 at most.
constexpr int kBwdThreads = 128, kBwdJ = 2;

// kBf16 is the type of dY and dYp, kBf16Buf that of Yp.
template <bool kBf16, bool kBf16Buf>
__global__ void __launch_bounds__(kBwdThreads) combine_bwd_kernel(const PermuteArgs a, int64_t V) {
  constexpr int N = Vec<kBf16>::kN, M = Vec<kBf16Buf>::kN, Q = N / M;      // Q vectors of Yp beside one of dY
  __shared__ float s_dot[kBwdThreads / 32][kMaxSlots];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint4* dy = static_cast<const uint4*>(a.src);
  const uint4* yp = static_cast<const uint4*>(a.yp);
  uint4* dst = static_cast<uint4*>(a.dst);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int row = lane < a.k ? static_cast<int>(slot_row(a, t, lane)) : -1;
    const float weight = row >= 0 ? __ldg(a.weights + t * a.k + lane) : 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += kBwdJ) {
      int r[kBwdJ];
      float w[kBwdJ], dot[kBwdJ];
#pragma unroll
      for (int j = 0; j < kBwdJ; ++j) {
        r[j] = __shfl_sync(kFull, row, (j0 + j) & 31);
        w[j] = __shfl_sync(kFull, weight, (j0 + j) & 31);
        if (j0 + j >= a.k) r[j] = -1;
        dot[j] = 0.0f;
      }
      for (int64_t v = threadIdx.x; v < V; v += blockDim.x) {
        uint4 q[kBwdJ][Q];
        float d[N];
#pragma unroll
        for (int j = 0; j < kBwdJ; ++j) {
#pragma unroll
          for (int u = 0; u < Q; ++u)
            if (r[j] >= 0) q[j][u] = __ldg(yp + (r[j] * V + v) * Q + u);
        }
        unpack<kBf16>(__ldg(dy + t * V + v), d);
#pragma unroll
        for (int j = 0; j < kBwdJ; ++j) {
          if (r[j] < 0) continue;
          float o[N];
#pragma unroll
          for (int u = 0; u < Q; ++u) {
            float y[M];
            unpack<kBf16Buf>(q[j][u], y);
#pragma unroll
            for (int i = 0; i < M; ++i) dot[j] = fmaf(d[u * M + i], y[i], dot[j]);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = w[j] * d[i];
          dst[r[j] * V + v] = pack<kBf16>(o);
        }
      }
#pragma unroll
      for (int j = 0; j < kBwdJ; ++j) {
        dot[j] = warp_sum(dot[j]);
        if (lane == 0 && j0 + j < a.k) s_dot[warp][j0 + j] = dot[j];
      }
    }
    __syncthreads();
    if (threadIdx.x < a.k) {
      float sum = 0.0f;
      for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) sum += s_dot[w][threadIdx.x];
      a.dweights[t * a.k + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

static unsigned perm_grid(int64_t tasks, const void* fn) {
  const int64_t need = (tasks + kPermThreads / 32 - 1) / (kPermThreads / 32);
  const int64_t most = static_cast<int64_t>(sm_count()) * blocks_per_sm(fn, kPermThreads, 0) * 4;
  return static_cast<unsigned>(need < most ? need : most);
}

template <int kU>
static cudaError_t dispatch_u(const PermuteArgs& a, int64_t V, cudaStream_t s) {
  const int strips = static_cast<int>((V + 32 * kU - 1) / (32 * kU));
  auto kern = dispatch_kernel<kU>;
  return launch_ex(kern, dim3(perm_grid(a.T * strips, reinterpret_cast<const void*>(kern))), dim3(kPermThreads), 0, s,
                   true, a, V, strips);
}

cudaError_t launch_dispatch(const PermuteArgs& a, cudaStream_t s) {
  const int64_t V = a.H / (a.xt == AVR_BF16 ? 8 : 4);
  return a.T * V <= kFewVectors ? dispatch_u<1>(a, V, s) : dispatch_u<4>(a, V, s);
}

template <bool kBf16, bool kBf16Out, bool kWeighted, int kU>
static cudaError_t combine_u(const PermuteArgs& a, int64_t V, cudaStream_t s) {
  const int strips = static_cast<int>((V + 32 * kU - 1) / (32 * kU));
  auto kern = combine_kernel<kBf16, kBf16Out, kWeighted, kU>;
  return launch_ex(kern, dim3(perm_grid(a.T * strips, reinterpret_cast<const void*>(kern))), dim3(kPermThreads), 0, s,
                   true, a, V, strips);
}

template <bool kBf16, bool kBf16Out, bool kWeighted>
static cudaError_t combine_t(const PermuteArgs& a, cudaStream_t s) {
  const int64_t V = a.H / Vec<kBf16>::kN;
  return a.T * V <= kFewVectors ? combine_u<kBf16, kBf16Out, kWeighted, 1>(a, V, s)
                                : combine_u<kBf16, kBf16Out, kWeighted, 4>(a, V, s);
}

cudaError_t launch_combine(const PermuteArgs& a, cudaStream_t s) {
  const bool bf16 = a.xt == AVR_BF16;
  if (a.weights == nullptr) return bf16 ? combine_t<true, true, false>(a, s) : combine_t<false, false, false>(a, s);
  if (a.f32_buffer && bf16) return combine_t<false, true, true>(a, s);
  return bf16 ? combine_t<true, true, true>(a, s) : combine_t<false, false, true>(a, s);
}

template <bool kBf16, bool kBf16Buf>
static cudaError_t combine_bwd_t(const PermuteArgs& a, cudaStream_t s) {
  auto kern = combine_bwd_kernel<kBf16, kBf16Buf>;
  const int64_t V = a.H / Vec<kBf16>::kN, passes = (V + kBwdThreads - 1) / kBwdThreads;
  const int threads = static_cast<int>(((V + passes - 1) / passes + 31) / 32 * 32);
  const int64_t most = static_cast<int64_t>(sm_count()) *
                       blocks_per_sm(reinterpret_cast<const void*>(kern), threads, 0) * 4;
  return launch_ex(kern, dim3(static_cast<unsigned>(a.T < most ? a.T : most)), dim3(threads), 0, s, true, a, V);
}

cudaError_t launch_combine_bwd(const PermuteArgs& a, cudaStream_t s) {
  if (a.xt != AVR_BF16) return combine_bwd_t<false, false>(a, s);
  return a.f32_buffer ? combine_bwd_t<true, false>(a, s) : combine_bwd_t<true, true>(a, s);
}

}  // namespace avr
