// The C ABI of the routing and 8-bit calls (declared in include/averis.h):
// host-side validation, workspace layout and the launch chains.
#include "route.h"

namespace avr {
namespace {

constexpr int64_t kMaxRows = kMaxDim - 511;      // so that a row coordinate rounded up to a tile stays an int32
bool rows_ok(int64_t l) { return l >= 0 && l <= kMaxRows; }
bool size16_ok(int64_t K) { return K > 0 && K % 16 == 0 && K <= kMaxRows; }
bool cap_ok(int64_t l_cap) { return rows_ok(l_cap) && l_cap % 128 == 0; }
bool slots_ok(int64_t T, int k) { return T >= 0 && k >= 1 && k <= kMaxSlots && T <= kMaxDim / k; }
bool experts_ok(int E) { return E >= 1 && E <= kMaxExperts; }

avr_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return AVR_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return AVR_ERR_MISALIGNED;
  return ws_bytes < need ? AVR_ERR_WORKSPACE_TOO_SMALL : AVR_OK;
}
uint32_t* status_of(void* ws) { return static_cast<uint32_t*>(ws); }

avr_status check_fp8(const avr_fp8* t, int64_t rows, int64_t K) {
  if (!t || !t->codes || !t->scales || t->rows != rows || t->K != K) return AVR_ERR_INVALID_ARG;
  return aligned16(t->codes) && aligned16(t->scales) ? AVR_OK : AVR_ERR_MISALIGNED;
}

// scratch of the linear calls after kScratch: the quantized row operand, or
// the two token-axis operands of the weight gradient, and before them the
// experts' tables (l_cap rows)
struct Fp8Layout {
  size_t seg = 0, block_expert = 0, order = 0, fits = 0;
  size_t q_codes = 0, q_scales = 0;                                        // [l, max(m, n)]
  size_t xt_codes = 0, xt_scales = 0, dt_codes = 0, dt_scales = 0;         // [m, L], [n, L]
  size_t total = 0;
};

Fp8Layout fp8_layout(int64_t l, int64_t m, int64_t n, int E) {
  Fp8Layout w;
  size_t off = kScratch;
  if (E > 0) {
    const size_t blocks = static_cast<size_t>(l / 128);
    w.seg = off;          off = align256(off + static_cast<size_t>(E) * sizeof(Fp8Seg));
    w.block_expert = off; off = align256(off + blocks * sizeof(int32_t));
    w.order = off;        off = align256(off + static_cast<size_t>(E) * sizeof(int32_t));
    w.fits = off;         off += 256;
  }
  const int64_t K = m > n ? m : n, L = blocks128(l) * 128;
  w.q_codes = off;
  w.q_scales = align256(w.q_codes + static_cast<size_t>(l) * static_cast<size_t>(K));
  const size_t rows_end = align256(w.q_scales + fp8_scales_bytes(l, K));
  w.xt_codes = off;
  w.xt_scales = align256(w.xt_codes + static_cast<size_t>(m) * static_cast<size_t>(L));
  w.dt_codes = align256(w.xt_scales + fp8_scales_bytes(m, L));
  w.dt_scales = align256(w.dt_codes + static_cast<size_t>(n) * static_cast<size_t>(L));
  const size_t tokens_end = align256(w.dt_scales + fp8_scales_bytes(n, L));
  w.total = rows_end > tokens_end ? rows_end : tokens_end;
  return w;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

Fp8Table table_at(void* ws, const Fp8Layout& w) {
  return Fp8Table{at<Fp8Seg>(ws, w.seg), at<int32_t>(ws, w.block_expert), at<int32_t>(ws, w.order),
                  at<int32_t>(ws, w.fits)};
}

Fp8QuantArgs quant_args(const void* X, avr_dtype xt, int64_t rows, int64_t K, uint8_t* codes, uint8_t* scales,
                        void* ws) {
  Fp8QuantArgs q;
  q.X = X;
  q.xt = xt;
  q.rows = rows;
  q.K = K;
  q.codes = codes;
  q.scales = scales;
  q.status = status_of(ws);
  return q;
}

Fp8GemmArgs gemm_args(const uint8_t* a_codes, const uint8_t* a_scales, int64_t a_rows, const uint8_t* b_codes,
                      const uint8_t* b_scales, int64_t b_rows, int64_t K, int64_t M, int64_t N, void* Y,
                      int64_t y_rows, avr_dtype yt, void* ws) {
  Fp8GemmArgs g;
  g.a_codes = a_codes;
  g.a_scales = a_scales;
  g.a_rows = a_rows;
  g.b_codes = b_codes;
  g.b_scales = b_scales;
  g.b_rows = b_rows;
  g.K = K;
  g.M = M;
  g.N = N;
  g.Y = Y;
  g.y_rows = y_rows;
  g.yt = yt;
  g.flags = at<uint32_t>(ws, WsLayout{}.tickets);
  g.status = status_of(ws);
  return g;
}

avr_status linear(const void* X, avr_dtype xt, int64_t l, int64_t K, int64_t N, int64_t m, int64_t n,
                  const avr_fp8* w, void* Y, avr_dtype yt, void* ws, size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(xt) || !dtype_ok(yt)) return AVR_ERR_INVALID_ARG;
  if (!rows_ok(l) || !size16_ok(m) || !size16_ok(n)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (l == 0) return AVR_OK;
  if (!X || !Y) return AVR_ERR_INVALID_ARG;
  AVR_TRY(check_fp8(w, N, K));
  if (!aligned16(X) || !aligned16(Y)) return AVR_ERR_MISALIGNED;
  const Fp8Layout lay = fp8_layout(l, m, n, 0);
  AVR_TRY(check_ws(ws, ws_bytes, lay.total));
  AVR_TRY(device_ok());
  if (fp8_skinny_applies(l, K, N))
    return cuda_status(launch_fp8_skinny({X, xt, l, K, N, w->codes, w->scales, Y, yt, status_of(ws)}, stream));
  uint8_t *codes = at<uint8_t>(ws, lay.q_codes), *scales = at<uint8_t>(ws, lay.q_scales);
  AVR_TRY(cuda_status(launch_fp8_quant(quant_args(X, xt, l, K, codes, scales, ws), stream)));
  return cuda_status(
      launch_fp8_gemm(gemm_args(codes, scales, l, w->codes, w->scales, N, K, l, N, Y, l, yt, ws), stream));
}

bool moe_sizes_ok(int64_t l_cap, int E, int64_t m, int64_t n) {
  return cap_ok(l_cap) && experts_ok(E) && size16_ok(m) && size16_ok(n) && m % 128 == 0 && n % 128 == 0 &&
         rows_ok(E * m) && rows_ok(E * n);
}

// Y rows of every expert from xq
avr_status moe_product(const uint8_t* codes, const uint8_t* scales, int64_t l_cap, int64_t K, int E,
                       const avr_fp8* w, int64_t N, const int32_t* counts, void* Y, avr_dtype yt, void* ws,
                       cudaStream_t s) {
  Fp8GemmArgs g = gemm_args(codes, scales, l_cap, w->codes, w->scales, E * N, K, l_cap, N, Y, l_cap, yt, ws);
  g.mode = Fp8GemmArgs::kRows;
  g.E = E;
  g.counts = counts;
  return cuda_status(launch_fp8_gemm(g, s));
}

avr_status moe_linear(const void* X, avr_dtype xt, int64_t l_cap, const int32_t* counts, int E, int64_t K, int64_t N,
                      int64_t m, int64_t n, const avr_fp8* w, void* Y, avr_dtype yt, void* ws, size_t ws_bytes,
                      avr_stream stream) {
  if (!dtype_ok(xt) || !dtype_ok(yt)) return AVR_ERR_INVALID_ARG;
  if (!moe_sizes_ok(l_cap, E, m, n)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (!counts || (l_cap > 0 && (!X || !Y))) return AVR_ERR_INVALID_ARG;
  AVR_TRY(check_fp8(w, E * N, K));
  if (!aligned16(X) || !aligned16(Y) || !aligned4(counts)) return AVR_ERR_MISALIGNED;
  const Fp8Layout lay = fp8_layout(l_cap, m, n, E);
  AVR_TRY(check_ws(ws, ws_bytes, lay.total));
  AVR_TRY(device_ok());
  const Fp8Table table = table_at(ws, lay);
  AVR_TRY(cuda_status(launch_fp8_table(counts, E, l_cap, table, status_of(ws), stream)));
  if (l_cap == 0) return AVR_OK;
  uint8_t *codes = at<uint8_t>(ws, lay.q_codes), *scales = at<uint8_t>(ws, lay.q_scales);
  Fp8QuantArgs q = quant_args(X, xt, l_cap, K, codes, scales, ws);
  q.table = &table;
  AVR_TRY(cuda_status(launch_fp8_quant(q, stream)));
  return moe_product(codes, scales, l_cap, K, E, w, N, counts, Y, yt, ws, stream);
}

// what the calls on the experts' buffer check alike; `buf`s may be null only when they have no rows
avr_status check_permute(const void* tokens, const void* buf, const void* row, avr_dtype xt, int64_t T, int k,
                         int64_t H, int64_t l_cap, void* ws, size_t ws_bytes) {
  if (!dtype_ok(xt)) return AVR_ERR_INVALID_ARG;
  if (!slots_ok(T, k) || H <= 0 || H % 8 || H > kMaxDim || !cap_ok(l_cap)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return AVR_OK;
  if (!tokens || !row || (!buf && l_cap > 0)) return AVR_ERR_INVALID_ARG;
  if (!aligned16(tokens) || !aligned16(buf) || !aligned4(row)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  return device_ok();
}

PermuteArgs permute_args(const void* src, void* dst, avr_dtype xt, int64_t T, int k, int64_t H, const int32_t* row,
                         int64_t l_cap, void* ws) {
  PermuteArgs a = {};
  a.src = src;
  a.dst = dst;
  a.row = row;
  a.xt = xt;
  a.T = T;
  a.H = H;
  a.l_cap = l_cap;
  a.k = k;
  a.status = status_of(ws);
  return a;
}

// f32_buffer: Yp is fp32 whatever the tokens' type yt
avr_status combine(const void* Yp, bool f32_buffer, avr_dtype yt, int64_t T, int k, int64_t H, const int32_t* row,
                   const float* weights, int64_t l_cap, void* Y, void* ws, size_t ws_bytes, avr_stream stream) {
  if (T > 0 && !weights) return AVR_ERR_INVALID_ARG;
  if (!aligned4(weights)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_permute(Y, Yp, row, yt, T, k, H, l_cap, ws, ws_bytes));
  if (T == 0) return AVR_OK;
  PermuteArgs a = permute_args(Yp, Y, yt, T, k, H, row, l_cap, ws);
  a.f32_buffer = f32_buffer;
  a.weights = weights;
  return cuda_status(launch_combine(a, stream));
}

avr_status combine_bwd(const void* dY, const void* Yp, bool f32_buffer, avr_dtype yt, int64_t T, int k, int64_t H,
                       const int32_t* row, const float* weights, int64_t l_cap, void* dYp, float* dweights, void* ws,
                       size_t ws_bytes, avr_stream stream) {
  if (T > 0 && (!weights || !dweights || (l_cap > 0 && !dYp))) return AVR_ERR_INVALID_ARG;
  if (!aligned4(weights) || !aligned4(dweights) || !aligned16(dYp)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_permute(dY, Yp, row, yt, T, k, H, l_cap, ws, ws_bytes));
  if (T == 0) return AVR_OK;
  PermuteArgs a = permute_args(dY, dYp, yt, T, k, H, row, l_cap, ws);
  a.yp = Yp;
  a.f32_buffer = f32_buffer;
  a.weights = weights;
  a.dweights = dweights;
  return cuda_status(launch_combine_bwd(a, stream));
}

}  // namespace
}  // namespace avr

using namespace avr;

extern "C" {

// ---------------------------------------------------------------------------
// routing
// ---------------------------------------------------------------------------
size_t moe_route_workspace_size(int64_t T, int k, int E) {
  if (!slots_ok(T, k) || !experts_ok(E)) return 0;
  return align256(kScratch + sort_scratch_ints(T * k, E) * sizeof(int32_t));
}

avr_status moe_route(const void* logits, avr_dtype lt, int64_t T, int E, int k, int norm, int32_t* ids,
                     float* weights, void* ws, size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(lt)) return AVR_ERR_INVALID_ARG;
  if (!slots_ok(T, k) || !experts_ok(E) || k > E) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return AVR_OK;
  if (!logits || !ids || !weights) return AVR_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned4(ids) || !aligned4(weights)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  return cuda_status(launch_route(logits, lt, T, E, k, norm != 0, ids, weights, status_of(ws), stream));
}

avr_status moe_route_bwd(const void* logits, avr_dtype lt, int64_t T, int E, int k, int norm, const int32_t* ids,
                         const float* weights, const float* dweights, void* dlogits, void* ws, size_t ws_bytes,
                         avr_stream stream) {
  if (!dtype_ok(lt)) return AVR_ERR_INVALID_ARG;
  if (!slots_ok(T, k) || !experts_ok(E) || k > E) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return AVR_OK;
  if ((!logits && !norm) || !ids || !weights || !dweights || !dlogits) return AVR_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(dlogits) || !aligned4(ids) || !aligned4(weights) || !aligned4(dweights))
    return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  return cuda_status(
      launch_route_bwd(logits, lt, T, E, k, norm != 0, ids, weights, dweights, dlogits, status_of(ws), stream));
}

avr_status moe_sort(const int32_t* ids, int64_t T, int k, int E, int64_t l_cap, int32_t* counts, int32_t* row,
                    void* ws, size_t ws_bytes, avr_stream stream) {
  if (!slots_ok(T, k) || !experts_ok(E) || !cap_ok(l_cap)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (!counts || (T > 0 && (!ids || !row))) return AVR_ERR_INVALID_ARG;
  if (!aligned4(ids) || !aligned4(counts) || !aligned4(row)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, moe_route_workspace_size(T, k, E)));
  AVR_TRY(device_ok());
  return cuda_status(launch_sort(ids, T * k, E, l_cap, counts, row, at<int32_t>(ws, kScratch), status_of(ws), stream));
}

avr_status moe_dispatch(const void* X, avr_dtype xt, int64_t T, int k, int64_t H, const int32_t* row, int64_t l_cap,
                        void* Xp, void* ws, size_t ws_bytes, avr_stream stream) {
  AVR_TRY(check_permute(X, Xp, row, xt, T, k, H, l_cap, ws, ws_bytes));
  if (T == 0) return AVR_OK;
  return cuda_status(launch_dispatch(permute_args(X, Xp, xt, T, k, H, row, l_cap, ws), stream));
}

avr_status moe_dispatch_bwd(const void* dXp, avr_dtype xt, int64_t T, int k, int64_t H, const int32_t* row,
                            int64_t l_cap, void* dX, void* ws, size_t ws_bytes, avr_stream stream) {
  AVR_TRY(check_permute(dX, dXp, row, xt, T, k, H, l_cap, ws, ws_bytes));
  if (T == 0) return AVR_OK;
  return cuda_status(launch_combine(permute_args(dXp, dX, xt, T, k, H, row, l_cap, ws), stream));
}

avr_status moe_combine(const void* Yp, avr_dtype yt, int64_t T, int k, int64_t H, const int32_t* row,
                       const float* weights, int64_t l_cap, void* Y, void* ws, size_t ws_bytes, avr_stream stream) {
  return combine(Yp, false, yt, T, k, H, row, weights, l_cap, Y, ws, ws_bytes, stream);
}

avr_status moe_combine_bwd(const void* dY, const void* Yp, avr_dtype yt, int64_t T, int k, int64_t H,
                           const int32_t* row, const float* weights, int64_t l_cap, void* dYp, float* dweights,
                           void* ws, size_t ws_bytes, avr_stream stream) {
  return combine_bwd(dY, Yp, false, yt, T, k, H, row, weights, l_cap, dYp, dweights, ws, ws_bytes, stream);
}

avr_status moe_combine_f32(const float* Yp, avr_dtype yt, int64_t T, int k, int64_t H, const int32_t* row,
                           const float* weights, int64_t l_cap, void* Y, void* ws, size_t ws_bytes,
                           avr_stream stream) {
  return combine(Yp, true, yt, T, k, H, row, weights, l_cap, Y, ws, ws_bytes, stream);
}

avr_status moe_combine_f32_bwd(const void* dY, const float* Yp, avr_dtype yt, int64_t T, int k, int64_t H,
                               const int32_t* row, const float* weights, int64_t l_cap, void* dYp, float* dweights,
                               void* ws, size_t ws_bytes, avr_stream stream) {
  return combine_bwd(dY, Yp, true, yt, T, k, H, row, weights, l_cap, dYp, dweights, ws, ws_bytes, stream);
}

// ---------------------------------------------------------------------------
// 8-bit linear layer
// ---------------------------------------------------------------------------
size_t avr_fp8_scales_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K <= 0 || K % 16) return 0;
  return fp8_scales_bytes(rows, K);
}

size_t fp8_workspace_size(int64_t l, int64_t m, int64_t n) {
  if (!rows_ok(l) || !size16_ok(m) || !size16_ok(n)) return 0;
  return fp8_layout(l, m, n, 0).total;
}

avr_status fp8_quant(const void* X, avr_dtype xt, int64_t rows, int64_t K, const avr_fp8* out, void* ws,
                     size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(xt)) return AVR_ERR_INVALID_ARG;
  if (!rows_ok(rows) || !size16_ok(K)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return AVR_OK;
  if (!X) return AVR_ERR_INVALID_ARG;
  AVR_TRY(check_fp8(out, rows, K));
  if (!aligned16(X)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  return cuda_status(launch_fp8_quant(quant_args(X, xt, rows, K, out->codes, out->scales, ws), stream));
}

avr_status fp8_quant_t(const void* X, avr_dtype xt, int64_t l, int64_t K, const avr_fp8* out, void* ws,
                       size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(xt)) return AVR_ERR_INVALID_ARG;
  if (!rows_ok(l) || !size16_ok(K)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (l == 0) return AVR_OK;
  if (!X) return AVR_ERR_INVALID_ARG;
  AVR_TRY(check_fp8(out, K, blocks128(l) * 128));
  if (!aligned16(X)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  return cuda_status(launch_fp8_quant_t(quant_args(X, xt, l, K, out->codes, out->scales, ws), nullptr, stream));
}

static avr_status quant_weights(const void* W, avr_dtype wt, int E, int64_t m, int64_t n, const avr_fp8* w_fwd,
                                const avr_fp8* w_dgrad, void* ws, size_t ws_bytes, avr_stream stream) {
  if (blocks128(m) > kFp8MaxWeightBlocks) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (!W) return AVR_ERR_INVALID_ARG;
  AVR_TRY(check_fp8(w_fwd, E * n, m));
  if (w_dgrad) AVR_TRY(check_fp8(w_dgrad, E * m, n));
  if (!aligned16(W)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  return cuda_status(launch_fp8_quant_weight(W, wt, E, m, n, w_fwd->codes, w_fwd->scales,
                                             w_dgrad ? w_dgrad->codes : nullptr, w_dgrad ? w_dgrad->scales : nullptr,
                                             status_of(ws), stream));
}

avr_status fp8_quant_weight(const void* W, avr_dtype wt, int64_t m, int64_t n, const avr_fp8* w_fwd,
                            const avr_fp8* w_dgrad, void* ws, size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(wt)) return AVR_ERR_INVALID_ARG;
  if (!size16_ok(m) || !size16_ok(n)) return AVR_ERR_UNSUPPORTED_SHAPE;
  return quant_weights(W, wt, 1, m, n, w_fwd, w_dgrad, ws, ws_bytes, stream);
}

avr_status fp8_gemm(const avr_fp8* a, const avr_fp8* b, void* Y, avr_dtype yt, void* ws, size_t ws_bytes,
                    avr_stream stream) {
  if (!a || !b || !dtype_ok(yt)) return AVR_ERR_INVALID_ARG;
  if (!rows_ok(a->rows) || !size16_ok(a->K) || !size16_ok(b->rows)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (a->rows == 0) return AVR_OK;
  if (!Y) return AVR_ERR_INVALID_ARG;
  AVR_TRY(check_fp8(a, a->rows, a->K));
  AVR_TRY(check_fp8(b, b->rows, a->K));
  if (!aligned16(Y)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  return cuda_status(launch_fp8_gemm(gemm_args(a->codes, a->scales, a->rows, b->codes, b->scales, b->rows, a->K,
                                               a->rows, b->rows, Y, a->rows, yt, ws), stream));
}

avr_status fp8_linear_fwd(const void* X, avr_dtype xt, int64_t l, int64_t m, int64_t n, const avr_fp8* w_fwd, void* Y,
                          avr_dtype yt, void* ws, size_t ws_bytes, avr_stream stream) {
  return linear(X, xt, l, m, n, m, n, w_fwd, Y, yt, ws, ws_bytes, stream);
}

avr_status fp8_linear_dgrad(const void* D, avr_dtype dt, int64_t l, int64_t m, int64_t n, const avr_fp8* w_dgrad,
                            void* dX, avr_dtype xt, void* ws, size_t ws_bytes, avr_stream stream) {
  return linear(D, dt, l, n, m, m, n, w_dgrad, dX, xt, ws, ws_bytes, stream);
}

avr_status fp8_linear_wgrad(const void* X, avr_dtype xt, const void* D, avr_dtype dt, int64_t l, int64_t m, int64_t n,
                            void* dW, avr_dtype wt, void* ws, size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(xt) || !dtype_ok(dt) || !dtype_ok(wt)) return AVR_ERR_INVALID_ARG;
  if (!rows_ok(l) || !size16_ok(m) || !size16_ok(n)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (!dW || (l > 0 && (!X || !D))) return AVR_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(D) || !aligned16(dW)) return AVR_ERR_MISALIGNED;
  const Fp8Layout lay = fp8_layout(l, m, n, 0);
  AVR_TRY(check_ws(ws, ws_bytes, lay.total));
  AVR_TRY(device_ok());
  if (l == 0)
    return cuda_status(cudaMemsetAsync(dW, 0, static_cast<size_t>(m) * static_cast<size_t>(n) *
                                                  (wt == AVR_BF16 ? 2 : 4), stream));
  uint8_t *xc = at<uint8_t>(ws, lay.xt_codes), *xs = at<uint8_t>(ws, lay.xt_scales);
  uint8_t *dc = at<uint8_t>(ws, lay.dt_codes), *ds = at<uint8_t>(ws, lay.dt_scales);
  const Fp8QuantArgs qx = quant_args(X, xt, l, m, xc, xs, ws), qd = quant_args(D, dt, l, n, dc, ds, ws);
  AVR_TRY(cuda_status(launch_fp8_quant_t(qx, &qd, stream)));
  return cuda_status(
      launch_fp8_gemm(gemm_args(xc, xs, m, dc, ds, n, blocks128(l) * 128, m, n, dW, m, wt, ws), stream));
}

// ---------------------------------------------------------------------------
// experts
// ---------------------------------------------------------------------------
size_t fp8_moe_workspace_size(int64_t l_cap, int64_t m, int64_t n, int E) {
  if (!moe_sizes_ok(l_cap, E, m, n)) return 0;
  return fp8_layout(l_cap, m, n, E).total;
}

avr_status fp8_moe_quant_weights(const void* W, avr_dtype wt, int E, int64_t m, int64_t n, const avr_fp8* w_fwd,
                                 const avr_fp8* w_dgrad, void* ws, size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(wt)) return AVR_ERR_INVALID_ARG;
  if (!moe_sizes_ok(0, E, m, n)) return AVR_ERR_UNSUPPORTED_SHAPE;
  return quant_weights(W, wt, E, m, n, w_fwd, w_dgrad, ws, ws_bytes, stream);
}

avr_status fp8_moe_dispatch(const void* X, avr_dtype xt, int64_t T, int k, int64_t K, const int32_t* row,
                            const avr_fp8* xq, void* ws, size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(xt) || !xq) return AVR_ERR_INVALID_ARG;
  if (!slots_ok(T, k) || !rows_ok(T) || !size16_ok(K) || K % 128 || !cap_ok(xq->rows)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return AVR_OK;
  if (!X || !row || xq->K != K) return AVR_ERR_INVALID_ARG;
  if (xq->rows > 0) AVR_TRY(check_fp8(xq, xq->rows, K));
  if (!aligned16(X) || !aligned4(row)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  Fp8QuantArgs q = quant_args(X, xt, T, K, xq->codes, xq->scales, ws);
  q.row = row;
  q.k = k;
  q.l_cap = xq->rows;
  return cuda_status(launch_fp8_quant(q, stream));
}

avr_status fp8_moe_gemm(const avr_fp8* xq, const int32_t* counts, int E, const avr_fp8* w, void* Y, avr_dtype yt,
                        void* ws, size_t ws_bytes, avr_stream stream) {
  if (!xq || !w || !dtype_ok(yt)) return AVR_ERR_INVALID_ARG;
  if (!experts_ok(E) || w->rows % E) return AVR_ERR_UNSUPPORTED_SHAPE;
  const int64_t l_cap = xq->rows, K = xq->K, N = w->rows / E;
  if (!moe_sizes_ok(l_cap, E, K, N)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (!counts || (l_cap > 0 && !Y)) return AVR_ERR_INVALID_ARG;
  if (l_cap > 0) AVR_TRY(check_fp8(xq, l_cap, K));
  AVR_TRY(check_fp8(w, E * N, K));
  if (!aligned16(Y) || !aligned4(counts)) return AVR_ERR_MISALIGNED;
  AVR_TRY(check_ws(ws, ws_bytes, kScratch));
  AVR_TRY(device_ok());
  if (l_cap == 0) return AVR_OK;
  return moe_product(xq->codes, xq->scales, l_cap, K, E, w, N, counts, Y, yt, ws, stream);
}

avr_status fp8_moe_linear_fwd(const void* X, avr_dtype xt, int64_t l_cap, const int32_t* counts, int E, int64_t m,
                              int64_t n, const avr_fp8* w_fwd, void* Y, avr_dtype yt, void* ws, size_t ws_bytes,
                              avr_stream stream) {
  return moe_linear(X, xt, l_cap, counts, E, m, n, m, n, w_fwd, Y, yt, ws, ws_bytes, stream);
}

avr_status fp8_moe_linear_dgrad(const void* D, avr_dtype dt, int64_t l_cap, const int32_t* counts, int E, int64_t m,
                                int64_t n, const avr_fp8* w_dgrad, void* dX, avr_dtype xt, void* ws, size_t ws_bytes,
                                avr_stream stream) {
  return moe_linear(D, dt, l_cap, counts, E, n, m, m, n, w_dgrad, dX, xt, ws, ws_bytes, stream);
}

avr_status fp8_moe_linear_wgrad(const void* X, avr_dtype xt, const void* D, avr_dtype dt, int64_t l_cap,
                                const int32_t* counts, int E, int64_t m, int64_t n, void* dW, avr_dtype wt, void* ws,
                                size_t ws_bytes, avr_stream stream) {
  if (!dtype_ok(xt) || !dtype_ok(dt) || !dtype_ok(wt)) return AVR_ERR_INVALID_ARG;
  if (!moe_sizes_ok(l_cap, E, m, n)) return AVR_ERR_UNSUPPORTED_SHAPE;
  if (!counts || !dW || (l_cap > 0 && (!X || !D))) return AVR_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(D) || !aligned16(dW) || !aligned4(counts)) return AVR_ERR_MISALIGNED;
  const Fp8Layout lay = fp8_layout(l_cap, m, n, E);
  AVR_TRY(check_ws(ws, ws_bytes, lay.total));
  AVR_TRY(device_ok());
  const Fp8Table table = table_at(ws, lay);
  AVR_TRY(cuda_status(launch_fp8_table(counts, E, l_cap, table, status_of(ws), stream)));
  if (l_cap == 0)
    return cuda_status(cudaMemsetAsync(dW, 0, static_cast<size_t>(E) * static_cast<size_t>(m) *
                                                  static_cast<size_t>(n) * (wt == AVR_BF16 ? 2 : 4), stream));
  uint8_t *xc = at<uint8_t>(ws, lay.xt_codes), *xs = at<uint8_t>(ws, lay.xt_scales);
  uint8_t *dc = at<uint8_t>(ws, lay.dt_codes), *ds = at<uint8_t>(ws, lay.dt_scales);
  Fp8QuantArgs qx = quant_args(X, xt, l_cap, m, xc, xs, ws), qd = quant_args(D, dt, l_cap, n, dc, ds, ws);
  qx.table = &table;
  qd.table = &table;
  AVR_TRY(cuda_status(launch_fp8_quant_t(qx, &qd, stream)));
  Fp8GemmArgs g = gemm_args(xc, xs, m, dc, ds, n, l_cap, m, n, dW, static_cast<int64_t>(E) * m, wt, ws);
  g.mode = Fp8GemmArgs::kTokens;
  g.E = E;
  g.table = &table;
  return cuda_status(launch_fp8_gemm(g, stream));
}

}  // extern "C"
