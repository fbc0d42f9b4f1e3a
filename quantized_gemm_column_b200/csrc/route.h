// Host-side interface of the routing kernels (route.cu) and the 8-bit ones
// (fp8_quant.cu, fp8_gemm.cu) for their C entry points (api_fp8.cu).
#pragma once

#include <atomic>

#include "internal.h"

namespace avr {

// A workspace of these calls starts like any other (status block, tickets:
// averis_check_status clears that much), so that one workspace serves all
// calls of the library; their scratch comes after it and is written by each
// call before it is read.
constexpr size_t kScratch = 256 + 4 * kMaxColTiles;
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int kMaxSlots = 32;        // k
constexpr int kMaxExperts = 1024;    // E

// ---------------- routing (route.cu) ----------------
cudaError_t launch_route(const void* logits, avr_dtype lt, int64_t T, int E, int k, int norm, int32_t* ids,
                         float* weights, uint32_t* status, cudaStream_t s);
cudaError_t launch_route_bwd(const void* logits, avr_dtype lt, int64_t T, int E, int k, int norm, const int32_t* ids,
                             const float* weights, const float* dweights, void* dlogits, uint32_t* status,
                             cudaStream_t s);

// chunks of slots that the sort's CTAs take, and the ints of its scratch
int sort_chunks(int64_t slots);
inline size_t sort_scratch_ints(int64_t slots, int E) {
  const int g = sort_chunks(slots);
  return g > 1 ? static_cast<size_t>(g) * static_cast<size_t>(E) : 0;
}
cudaError_t launch_sort(const int32_t* ids, int64_t slots, int E, int64_t l_cap, int32_t* counts, int32_t* row,
                        int32_t* scratch, uint32_t* status, cudaStream_t s);

struct PermuteArgs {
  const void* src;         // dispatch: X [T, H]; combine: Yp [l_cap, H]; combine_bwd: dY [T, H]
  const void* yp;          // combine_bwd: Yp [l_cap, H]
  void* dst;               // dispatch: Xp; combine: Y; combine_bwd: dYp
  const int32_t* row;      // [T, k]
  const float* weights;    // [T, k]; combine: null = all 1 (dispatch_bwd)
  float* dweights;         // combine_bwd
  avr_dtype xt;
  bool f32_buffer;         // combine, combine_bwd: Yp is fp32 whatever xt
  int64_t T, H, l_cap;
  int k;
  uint32_t* status;
};
cudaError_t launch_dispatch(const PermuteArgs& a, cudaStream_t s);
cudaError_t launch_combine(const PermuteArgs& a, cudaStream_t s);
cudaError_t launch_combine_bwd(const PermuteArgs& a, cudaStream_t s);

// ---------------- 8-bit blocks of 128 (fp8_quant.cu) ----------------
inline int64_t blocks128(int64_t x) { return (x + 127) / 128; }
// 512-byte scale atoms (128 rows x 4 blocks) along K
inline int64_t atoms128(int64_t K) { return (blocks128(K) + 3) / 4; }
inline size_t fp8_scales_bytes(int64_t rows, int64_t K) {
  return static_cast<size_t>(blocks128(rows)) * static_cast<size_t>(atoms128(K)) * 512;
}

// The experts' buffer as the quantizers and the weight gradients see it, from
// the counts: segments, and the expert of every 128-row block (-1 past the last).
struct Fp8Seg {
  int32_t row0, rows;
};
struct Fp8Table {
  Fp8Seg* seg;              // [E]
  int32_t* block_expert;    // [l_cap / 128]
  int32_t* order;           // [E] experts, the ones with the most tokens first
  int32_t* fits;            // 1 when the segments fit, else 0
};
cudaError_t launch_fp8_table(const int32_t* counts, int E, int64_t l_cap, const Fp8Table& t, uint32_t* status,
                             cudaStream_t s);

struct Fp8QuantArgs {
  const void* X;               // [rows, K]
  avr_dtype xt;
  int64_t rows, K;
  uint8_t* codes;
  uint8_t* scales;
  uint32_t* status;
  const Fp8Table* table = nullptr;   // grouped: only the rows that hold a token
  const int32_t* row = nullptr;      // dispatch: X [T = rows, K] to the buffer rows row[t, 0 .. k)
  int k = 0;
  int64_t l_cap = 0;
};
cudaError_t launch_fp8_quant(const Fp8QuantArgs& a, cudaStream_t s);
// along the tokens: X [rows, K] -> [K, L], L = rows rounded up to 128; b: a second tensor over the same tokens
cudaError_t launch_fp8_quant_t(const Fp8QuantArgs& a, const Fp8QuantArgs* b, cudaStream_t s);
// W [E][m][n] -> fwd [E n, m], dgrad [E m, n] (nullable codes); m in 65535 blocks at most
constexpr int64_t kFp8MaxWeightBlocks = 65535;
cudaError_t launch_fp8_quant_weight(const void* W, avr_dtype wt, int E, int64_t m, int64_t n, uint8_t* fwd_codes,
                                    uint8_t* fwd_scales, uint8_t* dg_codes, uint8_t* dg_scales, uint32_t* status,
                                    cudaStream_t s);

// ---------------- 8-bit product (fp8_gemm.cu) ----------------
// CTA pairs of a product; each has 16 flags in the workspace's tickets, zero between calls
constexpr int kFp8MaxPairs = 128;
static_assert(kFp8MaxPairs * 16 <= kMaxColTiles, "flags in the tickets");

struct Fp8GemmArgs {
  const uint8_t* a_codes;      // [a_rows, K]
  const uint8_t* a_scales;
  const uint8_t* b_codes;      // [b_rows, K]
  const uint8_t* b_scales;
  int64_t a_rows, b_rows, K;
  int64_t M, N;                // of one product
  void* Y;                     // [y_rows, N]
  int64_t y_rows;
  avr_dtype yt;
  uint32_t* flags;
  uint32_t* status;
  // one product; the row tiles of the experts' buffer, B = the experts stacked
  // (counts); or one product per expert along its tokens, Y = the experts
  // stacked (table)
  enum Mode { kDense, kRows, kTokens } mode = kDense;
  int E = 1;
  const int32_t* counts = nullptr;
  const Fp8Table* table = nullptr;
};
cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t s);
constexpr int kFp8MaxVisit = 48;     // blocks of K that one accumulation of an fp32 output spans
// the experts' products with few rows an expert (fp8_stream.cu): kRows
constexpr int64_t kStreamBlocks = 2;
bool fp8_stream_applies(const Fp8GemmArgs& a);
cudaError_t launch_fp8_stream(const Fp8GemmArgs& a, cudaStream_t s);
// clusters of two CTAs of `fn` that can be resident at once on the current
// device, kept per device in `cache` (zeros at first)
constexpr int kFp8CachedDevices = 64;
int fp8_resident_pairs(const void* fn, int threads, size_t smem, std::atomic<int>* cache);

// ---------------- 8-bit linear layer of a few tokens (fp8_skinny.cu) ----------------
// Y [l, N] = Q(X) w^T, w [N, K]
struct Fp8SkinnyArgs {
  const void* X;
  avr_dtype xt;
  int64_t l, K, N;
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  void* Y;
  avr_dtype yt;
  uint32_t* status;
};
bool fp8_skinny_applies(int64_t l, int64_t K, int64_t N);
cudaError_t launch_fp8_skinny(const Fp8SkinnyArgs& a, cudaStream_t s);

}  // namespace avr
