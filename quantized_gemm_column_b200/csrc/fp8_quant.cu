// Quantizers of the 8-bit linear layer: E4M3 codes with a power-of-two scale
// per block of 128 (the rule is in include/averis.h), written in the layouts
// the block-scaled product reads.
//
// Every element is read once and its byte written once: 3 bytes of memory
// traffic an element from bf16, 5 from fp32, and a few instructions; the
// kernels are bound by memory once those few are few enough: magnitudes are
// compared two bf16 at a time, products taken two fp32 at a time.  The maxima
// keep a NaN, and the bits of the result order as it does, so the exponent and
// the non-finite check fall out of them.
#include "fp8_common.cuh"
#include "route.h"
#include "strips.cuh"

namespace avr {

using namespace fp8;

// ---------------------------------------------------------------------------
// segment table of the experts' buffer (one CTA)
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 1024;

__global__ void __launch_bounds__(kTableThreads) fp8_table_kernel(const int32_t* counts, int E, int64_t l_cap,
                                                                  const Fp8Table t, uint32_t* status) {
  __shared__ int32_t s_rows[kMaxExperts], s_blk[kMaxExperts];   // rows; ends in blocks
  __shared__ uint64_t s_warp[32];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t n = tid < E ? __ldg(counts + tid) : 0;
  const bool bad = n < 0 || n > l_cap;
  const bool any_bad = __syncthreads_or(bad) != 0;
  const uint64_t blk = bad ? 0 : (static_cast<uint64_t>(n) + 127) / 128;
  uint64_t x = blk;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint64_t y = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t z = __shfl_up_sync(kFull, y, o);
      if (lane >= o) y += z;
    }
    s_warp[lane] = y;
  }
  __syncthreads();
  if (warp > 0) x += s_warp[warp - 1];
  const int64_t n_blocks = l_cap / 128;
  const bool fits = !any_bad && static_cast<int64_t>(s_warp[31]) <= n_blocks;
  const int32_t blocks = fits ? static_cast<int32_t>(s_warp[31]) : 0;
  if (tid < E) s_rows[tid] = n;
  if (tid < E && fits) {
    s_blk[tid] = static_cast<int32_t>(x);
    t.seg[tid] = Fp8Seg{static_cast<int32_t>(128 * (x - blk)), n};
  }
  if (tid == 0) {
    *t.fits = fits ? 1 : 0;
    if (!fits) raise_status(status, AVR_ERR_INVALID_ARG);
  }
  __syncthreads();
  if (tid < E && fits) {
    int rank = 0;
    for (int e = 0; e < E; ++e) rank += s_rows[e] > n || (s_rows[e] == n && e < tid) ? 1 : 0;
    t.order[rank] = tid;
  }
  // the first expert whose end lies past i
  auto find = [&](const int32_t* end, int32_t i) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (end[mid] > i)
        hi = mid;
      else
        lo = mid + 1;
    }
    return lo;
  };
  for (int32_t b = tid; b < n_blocks; b += kTableThreads) t.block_expert[b] = b < blocks ? find(s_blk, b) : -1;
}

cudaError_t launch_fp8_table(const int32_t* counts, int E, int64_t l_cap, const Fp8Table& t, uint32_t* status,
                             cudaStream_t s) {
  return launch_ex(fp8_table_kernel, dim3(1), dim3(kTableThreads), 0, s, true, counts, E, l_cap, t, status);
}

// ---------------------------------------------------------------------------
// along K: a warp takes kRows rows x 512 columns, 16 columns a lane, so that
// eight lanes share a block and the warp's four scale bytes are one word of an
// atom.  kRows rows' loads are in flight at once, four of bf16 or two of fp32
// (64 bytes a lane and row), with four blocks an SM: 16384 x 6144 bf16 takes
// 46 us (6.6 TB/s), with two rows 50; 4133 x 2000 fp32 8.4 us, with four 17
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;
constexpr int kQWarps = kQThreads / 32;

enum class Rows { kAll, kGrouped, kDispatch };

template <bool kBf16, Rows kMode, int kRows>
__global__ void __launch_bounds__(kQThreads, 4) fp8_quant_kernel(const Fp8QuantArgs a, const Fp8Table t, int64_t rows_pad,
                                                              int strips) {
  constexpr int N = In<kBf16>::kN, Q = 16 / N;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  if (kMode == Rows::kGrouped && __ldcg(t.fits) == 0) return;
  const int lane = threadIdx.x & 31;
  const uint4* X = static_cast<const uint4*>(a.X);
  const int64_t V = a.K / N;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kQWarps;
  const int64_t tasks = (rows_pad / kRows) * strips;
  bool bad = false;
  for (StripWalk at(static_cast<int64_t>(blockIdx.x) * kQWarps + (threadIdx.x >> 5), warps, tasks, strips); at.more();
       at.step()) {
    const int strip = at.strip;
    const int64_t r0 = at.row * kRows;
    const int64_t col = static_cast<int64_t>(strip) * 512 + 16 * lane;
    int64_t end = a.rows;
    if (kMode == Rows::kGrouped) {        // a task lies in one 128-row block, so in one segment
      const int e = __ldcg(t.block_expert + r0 / 128);
      if (e < 0) break;                   // past the last segment, and so is all that follows
      const int2 sg = __ldcg(reinterpret_cast<const int2*>(t.seg + e));
      end = static_cast<int64_t>(sg.x) + sg.y;
    }
    uint4 q[kRows][Q];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int u = 0; u < Q; ++u)
        q[i][u] = (r0 + i < end && col < a.K) ? __ldg(X + (r0 + i) * V + col / N + u) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = r0 + i;
      if (kMode != Rows::kAll && r >= end) break;      // the whole warp
      uint4 codes;
      uint32_t word;
      bool nonfinite = false;
      quant_strip<kBf16>(q[i], &codes, &word, &nonfinite);
      auto put = [&](int64_t dst) {
        if (col < a.K) *reinterpret_cast<uint4*>(a.codes + dst * a.K + col) = codes;
        if (lane == 0) *reinterpret_cast<uint32_t*>(a.scales + scale_at(dst, 4 * strip, strips)) = word;
      };
      if (kMode == Rows::kDispatch) {
        for (int j = 0; j < a.k; ++j) {
          const int32_t dst = __ldg(a.row + r * a.k + j);
          if (dst >= a.l_cap) raise_status(a.status, AVR_ERR_INVALID_ARG);
          if (dst >= 0 && dst < a.l_cap) {
            put(dst);
            bad |= nonfinite;             // a token without a row may hold anything
          }
        }
        continue;
      }
      bad |= nonfinite;
      if (r < end) {
        put(r);
      } else if (lane == 0) {             // rows up to the next multiple of 128: zero scales
        *reinterpret_cast<uint32_t*>(a.scales + scale_at(r, 4 * strip, strips)) = 0u;
      }
    }
  }
  if (bad) raise_status(a.status, AVR_ERR_NONFINITE);
}

template <bool kBf16, Rows kMode, int kRows>
static cudaError_t quant_t(const Fp8QuantArgs& a, int64_t rows_pad, cudaStream_t s) {
  auto kern = fp8_quant_kernel<kBf16, kMode, kRows>;
  const int strips = static_cast<int>((a.K + 511) / 512);
  const int64_t need = (rows_pad / kRows * strips + kQWarps - 1) / kQWarps;
  const int64_t most = static_cast<int64_t>(sm_count()) *
                       blocks_per_sm(reinterpret_cast<const void*>(kern), kQThreads, 0) * 4;
  const Fp8Table t = a.table ? *a.table : Fp8Table{};
  return launch_ex(kern, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(kQThreads), 0, s, true, a, t,
                   rows_pad, strips);
}

cudaError_t launch_fp8_quant(const Fp8QuantArgs& a, cudaStream_t s) {
  const int64_t pad = blocks128(a.rows) * 128;
  if (a.row != nullptr)
    return a.xt == AVR_BF16 ? quant_t<true, Rows::kDispatch, 1>(a, a.rows, s)
                            : quant_t<false, Rows::kDispatch, 1>(a, a.rows, s);
  if (a.table != nullptr)
    return a.xt == AVR_BF16 ? quant_t<true, Rows::kGrouped, 4>(a, pad, s) : quant_t<false, Rows::kGrouped, 2>(a, pad, s);
  return a.xt == AVR_BF16 ? quant_t<true, Rows::kAll, 4>(a, pad, s) : quant_t<false, Rows::kAll, 2>(a, pad, s);
}

// ---------------------------------------------------------------------------
// along the tokens: a CTA takes 128 tokens x 8 vectors of features (64 bf16,
// 32 fp32).  A thread holds four consecutive tokens of one vector, so its
// codes of a feature are one word of the transposed tile; the tile goes
// through shared memory (rows of 33 words) and out as full 128-byte lines.
// 16384 x 6144 bf16: 54 us (5.6 TB/s).
// ---------------------------------------------------------------------------
template <bool kBf16>
__device__ __forceinline__ void quant_tokens(const Fp8QuantArgs& a, const Fp8Table& t, int64_t L, int64_t atoms,
                                             unsigned ftile, int64_t c) {
  constexpr int N = In<kBf16>::kN, F = 8 * N;
  __shared__ uint32_t s_max[kQWarps][32];            // maxima, a word as in the input
  __shared__ uint32_t s_byte[F];
  __shared__ uint32_t s_tile[F][33];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t f0 = static_cast<int64_t>(ftile) * F;
  int64_t end = a.rows;
  if (a.table != nullptr) {
    if (__ldcg(t.fits) == 0) return;
    const int e = __ldcg(t.block_expert + c);
    if (e < 0) return;
    const int2 sg = __ldcg(reinterpret_cast<const int2*>(t.seg + e));
    end = static_cast<int64_t>(sg.x) + sg.y;
  }
  const int v = tid & 7, g = tid >> 3;               // vector, group of four tokens
  const uint4* X = static_cast<const uint4*>(a.X);
  const int64_t V = a.K / N, vec = f0 / N + v;
  uint4 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = c * 128 + 4 * g + i;
    q[i] = (r < end && vec < V) ? __ldg(X + r * V + vec) : make_uint4(0u, 0u, 0u, 0u);
  }
  // a word is one fp32 feature or two bf16 ones
#pragma unroll
  for (int c4 = 0; c4 < 4; ++c4) {
    uint32_t m = abs_max<kBf16>(abs_max<kBf16>((&q[0].x)[c4], (&q[1].x)[c4]),
                                abs_max<kBf16>((&q[2].x)[c4], (&q[3].x)[c4]));
    m = abs_max<kBf16>(m, __shfl_xor_sync(kFull, m, 8));
    m = abs_max<kBf16>(m, __shfl_xor_sync(kFull, m, 16));
    if (lane < 8) s_max[warp][4 * v + c4] = m;
  }
  __syncthreads();
  bool bad = false;
  if (tid < F) {
    uint32_t top = 0;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      const uint32_t m = s_max[w][kBf16 ? tid / 2 : tid];
      top = max(top, kBf16 ? ((tid & 1) ? m & 0xFFFF0000u : m << 16) : m);
    }
    bad = top >= kInfBits;
    const uint32_t byte = scale_byte(top);
    s_byte[tid] = byte;
    const int64_t j = f0 + tid, at = scale_at(j, c, atoms);
    a.scales[at] = static_cast<uint8_t>(j < a.K ? byte : 0u);
    if (c == L / 128 - 1)                            // the atom's blocks past the last
      for (int64_t z = c + 1; z < 4 * atoms; ++z) a.scales[scale_at(j, z, atoms)] = 0;
  }
  if (bad) raise_status(a.status, AVR_ERR_NONFINITE);
  __syncthreads();
#pragma unroll
  for (int f = 0; f < N; ++f) {
    s_tile[N * v + f][g] = e4m3x4(value_of<kBf16>(q[0], f), value_of<kBf16>(q[1], f), value_of<kBf16>(q[2], f),
                                  value_of<kBf16>(q[3], f), inv_scale(s_byte[N * v + f]));
  }
  __syncthreads();
  for (int f = warp; f < F; f += kQWarps)
    if (f0 + f < a.K) *reinterpret_cast<uint32_t*>(a.codes + (f0 + f) * L + c * 128 + 4 * lane) = s_tile[f][lane];
}

// Feature tiles are the grid's x: they share the tokens' rows.  The blocks are
// short, so a division of the block index would show (54 us become 58).
template <bool kBf16>
__global__ void __launch_bounds__(kQThreads) fp8_quant_tokens_kernel(const Fp8QuantArgs a, const Fp8Table t,
                                                                     int64_t L, int64_t atoms) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int64_t c = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
  if (c * 128 < L) quant_tokens<kBf16>(a, t, L, atoms, blockIdx.x, c);
}

// two tensors over the same tokens: ftiles0 feature tiles of the first, then the second's
template <bool kBf16>
__global__ void __launch_bounds__(kQThreads)
    fp8_quant_tokens2_kernel(const Fp8QuantArgs a0, const Fp8QuantArgs a1, const Fp8Table t, int64_t L, int64_t atoms,
                             unsigned ftiles0) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int64_t c = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
  if (c * 128 >= L) return;
  if (blockIdx.x < ftiles0)
    quant_tokens<kBf16>(a0, t, L, atoms, blockIdx.x, c);
  else
    quant_tokens<kBf16>(a1, t, L, atoms, blockIdx.x - ftiles0, c);
}

// Two tensors in one launch save the second's start and end, about 2 us, which
// counts while they are small: 3300 blocks of 4133 tokens fp32 13 us, in two
// launches 16; larger ones go one after the other.
constexpr int64_t kTwoBlocks = 8192;

cudaError_t launch_fp8_quant_t(const Fp8QuantArgs& a, const Fp8QuantArgs* b, cudaStream_t s) {
  const int F = a.xt == AVR_BF16 ? 64 : 32;
  const int64_t L = blocks128(a.rows) * 128;
  const int64_t ftiles0 = blocks128(a.K) * 128 / F, ftiles = ftiles0 + (b ? blocks128(b->K) * 128 / F : 0);
  const int64_t grid = ftiles * (L / 128);
  if (b != nullptr && (b->xt != a.xt || grid > kTwoBlocks)) {
    cudaError_t e = launch_fp8_quant_t(a, nullptr, s);
    return e != cudaSuccess ? e : launch_fp8_quant_t(*b, nullptr, s);
  }
  const Fp8Table t = a.table ? *a.table : Fp8Table{};
  const int64_t blocks = L / 128, z = (blocks + 65534) / 65535;        // at most 2^24 blocks
  const dim3 g(static_cast<unsigned>(ftiles), static_cast<unsigned>((blocks + z - 1) / z), static_cast<unsigned>(z));
  const dim3 threads(kQThreads);
  if (b == nullptr) {
    auto kern = a.xt == AVR_BF16 ? fp8_quant_tokens_kernel<true> : fp8_quant_tokens_kernel<false>;
    return launch_ex(kern, g, threads, 0, s, true, a, t, L, atoms128(L));
  }
  auto kern = a.xt == AVR_BF16 ? fp8_quant_tokens2_kernel<true> : fp8_quant_tokens2_kernel<false>;
  return launch_ex(kern, g, threads, 0, s, true, a, *b, t, L, atoms128(L), static_cast<unsigned>(ftiles0));
}

// ---------------------------------------------------------------------------
// weights: a CTA takes one 128 x 128 block and writes it both ways round, the
// transposed codes through shared memory.  A block loads, then computes, then
// stores, so it takes four on an SM to keep memory busy: 64 x 2048 x 1024 bf16
// in 84 us (6.4 TB/s); 114 with the registers for three
// ---------------------------------------------------------------------------
template <bool kBf16>
__global__ void __launch_bounds__(kQThreads, kBf16 ? 4 : 2)
    fp8_quant_weight_kernel(const void* W, int64_t m, int64_t n, uint8_t* fwd_codes, uint8_t* fwd_scales,
                            uint8_t* dg_codes, uint8_t* dg_scales, int64_t atoms_m, int64_t atoms_n, uint32_t* status) {
  constexpr int N = In<kBf16>::kN, kCols = 128 / N;    // vectors of a row: 16 (bf16) or 32
  constexpr int kGroups = kQThreads / kCols;           // row groups: 16 or 8
  constexpr int R = 128 / kGroups;                     // consecutive rows of a thread: 8 or 16
  __shared__ uint32_t s_max[kQWarps];
  __shared__ uint32_t s_tile[128][33];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t bns = gridDim.x, bms = gridDim.y;
  const int64_t bn = blockIdx.x, bm = blockIdx.y, e = blockIdx.z;
  const int v = tid % kCols, g = tid / kCols;
  const uint4* X = static_cast<const uint4*>(W) + e * m * (n / N);
  const int64_t V = n / N, vec = bn * kCols + v;
  uint4 q[R];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = bm * 128 + R * g + i;
    q[i] = (r < m && vec < V) ? __ldg(X + r * V + vec) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) top = abs_max<kBf16>(top, abs_max<kBf16>(q[i]));
  top = __reduce_max_sync(kFull, amax_bits<kBf16>(top));
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQWarps; ++w) top = max(top, s_max[w]);
  if (top >= kInfBits && tid == 0) raise_status(status, AVR_ERR_NONFINITE);
  const uint32_t byte = scale_byte(top);
  const float inv = inv_scale(byte);
  // rows of this thread, N codes each
#pragma unroll
  for (int i4 = 0; i4 < R / 4; ++i4) {
    uint32_t w[4][N / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int b = 0; b < N / 4; ++b) {
        float f[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = value_of<kBf16>(q[4 * i4 + i], 4 * b + x);
        w[i][b] = e4m3x4(f[0], f[1], f[2], f[3], inv);
      }
      const int64_t r = bm * 128 + R * g + 4 * i4 + i;
      if (dg_codes != nullptr && r < m && vec < V) {
        uint8_t* dst = dg_codes + (e * m + r) * n + vec * N;
        if (N == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(w[i][0], w[i][N / 4 - 1]);
        else
          *reinterpret_cast<uint32_t*>(dst) = w[i][0];
      }
    }
#pragma unroll
    for (int b = 0; b < N / 4; ++b) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {                    // feature 4 b + x: four rows' codes as one word
        const uint32_t lo = __byte_perm(w[0][b], w[1][b], x | ((x + 4) << 4));
        const uint32_t hi = __byte_perm(w[2][b], w[3][b], x | ((x + 4) << 4));
        s_tile[N * v + 4 * b + x][(R * g) / 4 + i4] = (lo & 0xFFFFu) | (hi << 16);
      }
    }
  }
  __syncthreads();
  // w_fwd: feature rows of m codes (m % 16 == 0, so a word is wholly inside or outside)
  for (int f = warp; f < 128; f += kQWarps)
    if (bn * 128 + f < n && bm * 128 + 4 * lane < m)
      *reinterpret_cast<uint32_t*>(fwd_codes + (e * n + bn * 128 + f) * m + bm * 128 + 4 * lane) = s_tile[f][lane];
  if (tid < 128) {
    // experts are stacked by whole 128-row groups (E > 1 needs m and n in multiples of 128)
    const int64_t j = e * n + bn * 128 + tid;
    fwd_scales[scale_at(j, bm, atoms_m)] = static_cast<uint8_t>(bn * 128 + tid < n ? byte : 0u);
    if (bm == bms - 1)
      for (int64_t z = bm + 1; z < 4 * atoms_m; ++z) fwd_scales[scale_at(j, z, atoms_m)] = 0;
    if (dg_codes != nullptr) {
      const int64_t i = e * m + bm * 128 + tid;
      dg_scales[scale_at(i, bn, atoms_n)] = static_cast<uint8_t>(bm * 128 + tid < m ? byte : 0u);
      if (bn == bns - 1)
        for (int64_t z = bn + 1; z < 4 * atoms_n; ++z) dg_scales[scale_at(i, z, atoms_n)] = 0;
    }
  }
}

cudaError_t launch_fp8_quant_weight(const void* W, avr_dtype wt, int E, int64_t m, int64_t n, uint8_t* fwd_codes,
                                    uint8_t* fwd_scales, uint8_t* dg_codes, uint8_t* dg_scales, uint32_t* status,
                                    cudaStream_t s) {
  if (blocks128(m) > kFp8MaxWeightBlocks) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks128(n)), static_cast<unsigned>(blocks128(m)), static_cast<unsigned>(E));
  auto kern = wt == AVR_BF16 ? fp8_quant_weight_kernel<true> : fp8_quant_weight_kernel<false>;
  return launch_ex(kern, grid, dim3(kQThreads), 0, s, true, W, m, n, fwd_codes, fwd_scales,
                   dg_codes, dg_scales, atoms128(m), atoms128(n), status);
}

}  // namespace avr
