// The 8-bit linear layer for a few tokens (l <= 8): quantizer and product in
// one kernel on the CUDA cores.
//
// With a handful of rows the product is a pass over the weights' N K bytes and
// the rest is latency: a quantizer, a launch between, and tensor-core tiles
// that are 256 rows high.  Here every block quantizes the tokens for itself (X
// is l K elements, from L2) into shared memory, as the codes' values in fp16
// (exact) and scale bytes, while its first weights are on the way.  A warp
// takes R rows of W at a time, 16 codes a lane; a code pair becomes two fp16
// in one instruction and each product is exact in an fp32 fma.  The 16
// products of a lane lie in one block of 128, so the power-of-two scales
// multiply their sum once.  The sum over lanes is a shuffle tree: a fixed order.
#include "fp8_common.cuh"
#include "route.h"

namespace avr {

using namespace fp8;

namespace {

constexpr int kSkThreads = 256;
constexpr int kSkWarps = kSkThreads / 32;

// two E4M3 codes -> two fp16, exact
__device__ __forceinline__ uint32_t f16x2_of(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
// c + a.lo b.lo + a.hi b.hi, exact products, fp32 sums
__device__ __forceinline__ float fma2(uint32_t a, uint32_t b, float c) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return fmaf(x.y, y.y, fmaf(x.x, y.x, c));
}

}  // namespace

// R rows a warp, their codes of D strips (512 columns) in flight
template <int L, int R, int D>
__global__ void __launch_bounds__(kSkThreads, L <= 2 ? 3 : 2)
    fp8_skinny_kernel(const void* X, int bf16_in, int l, int64_t K, int64_t N, const uint8_t* w_codes,
                      const uint8_t* w_scales, void* Y, int bf16_out, int strips, uint32_t* status) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int64_t Kp = static_cast<int64_t>(strips) * 512;
  __half* xs = reinterpret_cast<__half*>(smem);                              // [L][Kp]
  uint8_t* sx = smem + static_cast<size_t>(L) * Kp * 2;                      // [L][4 strips]
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * kSkWarps + warp) * R;
  uint4 w[D][R];
  uint32_t sw[D][R];
  auto load = [&](int s, uint4 (&wd)[R], uint32_t (&sd)[R]) {
    const int64_t col = static_cast<int64_t>(s) * 512 + 16 * lane;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      wd[r] = make_uint4(0u, 0u, 0u, 0u);
      sd[r] = 0u;
      if (n0 + r < N && s < strips) {
        if (col < K) wd[r] = __ldg(reinterpret_cast<const uint4*>(w_codes + (n0 + r) * K + col));
        sd[r] = __ldg(reinterpret_cast<const uint32_t*>(w_scales + scale_at(n0 + r, 4 * s, strips)));
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, w[d], sw[d]);

  bool bad = false;
  for (int task = warp; task < L * strips; task += kSkWarps) {
    const int t = task / strips, s = task % strips;
    const int64_t col = static_cast<int64_t>(s) * 512 + 16 * lane;
    uint4 codes;
    uint32_t word;
    const bool in = t < l && col < K;
    if (bf16_in) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(X) + t * K + col);
      uint4 q[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) q[u] = in ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
      quant_strip<true>(q, &codes, &word, &bad);
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const float*>(X) + t * K + col);
      uint4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) q[u] = in ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
      quant_strip<false>(q, &codes, &word, &bad);
    }
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    uint4* dst = reinterpret_cast<uint4*>(xs + t * Kp + col);
    dst[0] = make_uint4(f16x2_of(c[0] & 0xFFFFu), f16x2_of(c[0] >> 16), f16x2_of(c[1] & 0xFFFFu), f16x2_of(c[1] >> 16));
    dst[1] = make_uint4(f16x2_of(c[2] & 0xFFFFu), f16x2_of(c[2] >> 16), f16x2_of(c[3] & 0xFFFFu), f16x2_of(c[3] >> 16));
    if (lane < 4) sx[(t * strips + s) * 4 + lane] = static_cast<uint8_t>(word >> (8 * lane));
  }
  if (bad) raise_status(status, AVR_ERR_NONFINITE);
  __syncthreads();

  float acc[R][L];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int t = 0; t < L; ++t) acc[r][t] = 0.0f;
  }
  for (int s0 = 0; s0 < strips; s0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int s = s0 + d;
      if (s >= strips) break;
      uint32_t wf[R][8], wb[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t c[4] = {w[d][r].x, w[d][r].y, w[d][r].z, w[d][r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wf[r][2 * i] = f16x2_of(c[i] & 0xFFFFu);
          wf[r][2 * i + 1] = f16x2_of(c[i] >> 16);
        }
        wb[r] = (sw[d][r] >> (8 * (lane >> 3))) & 0xFFu;
      }
      load(s + D, w[d], sw[d]);
      const int64_t col = static_cast<int64_t>(s) * 512 + 16 * lane;
#pragma unroll
      for (int t = 0; t < L; ++t) {
        const uint4 a = *reinterpret_cast<const uint4*>(xs + t * Kp + col);
        const uint4 b = *reinterpret_cast<const uint4*>(xs + t * Kp + col + 8);
        const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const uint32_t xb = sx[(t * strips + s) * 4 + (lane >> 3)];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p0 = fma2(wf[r][i], x[i], p0);
            p1 = fma2(wf[r][4 + i], x[4 + i], p1);
          }
          // 2^(xb + wb - 254) as two halves: what comes between lies between the
          // lane's sum and the scaled one, so nothing is lost that those can hold
          const uint32_t e = xb + wb[r], h = e >> 1;
          acc[r][t] = fmaf((p0 + p1) * __uint_as_float(h << 23), __uint_as_float((e - h) << 23), acc[r][t]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int t = 0; t < L; ++t) {
      float v = acc[r][t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
      if (lane == t && t < l && n0 + r < N) {
        const int64_t at = static_cast<int64_t>(t) * N + n0 + r;
        if (bf16_out)
          static_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(v);
        else
          static_cast<float*>(Y)[at] = v;
      }
    }
  }
}

// The tokens a kernel is compiled for.
static int skinny_tokens(int64_t l) { return l <= 1 ? 1 : l <= 2 ? 2 : l <= 4 ? 4 : 8; }

bool fp8_skinny_applies(int64_t l, int64_t K, int64_t N) {
  if (l > 8) return false;
  const int64_t L = skinny_tokens(l);
  if (L * ((K + 511) / 512) * 512 > 48 * 1024) return false;      // the tokens in shared memory
  // This kernel's time goes as L N K, the quantizer's and the product's as K
  // (one tile of rows whatever l).  us on the device, l = 1, 2, 4, 8 / theirs
  // (| where the rule changes over):
  //   1024 -> 6144   4.1   5.1   7.3 | 12   /  8.6
  //   4096 -> 4096   8.5  11.8  13.1 | 22   / 16.3
  //    512 -> 8192   4.2   5.0   6.4 |  9.9 /  7.4
  //   1024 -> 3584   3.7   4.4   4.7   7.7 |/  8.3
  //   2048 -> 2048   3.9   4.9   5.5   9.2 |/ 10.9
  //   8192 -> 1024   6.8   8.5  11.4  26.1 |/ 26.1
  //   6144 -> 1024   5.7   6.9   9.1  15.3 |/ 21
  //   1024 -> 1024   1.9   2.1   2.5   3.9 |/  7.9
  return L * N < (20000000 + 12000 * K) / K;
}

template <int L, int R, int D>
static cudaError_t skinny_t(const Fp8SkinnyArgs& a, cudaStream_t s) {
  const int strips = static_cast<int>((a.K + 511) / 512);
  const size_t smem = static_cast<size_t>(L) * strips * 512 * 2 + static_cast<size_t>(L) * strips * 4;
  auto kern = fp8_skinny_kernel<L, R, D>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = (a.N + kSkWarps * R - 1) / (kSkWarps * R);
  return launch_ex(kern, dim3(static_cast<unsigned>(grid)), dim3(kSkThreads), smem, s, true, a.X,
                   a.xt == AVR_BF16 ? 1 : 0, static_cast<int>(a.l), a.K, a.N, a.w_codes, a.w_scales, a.Y,
                   a.yt == AVR_BF16 ? 1 : 0, strips, a.status);
}

template <int L>
static cudaError_t skinny_l(const Fp8SkinnyArgs& a, cudaStream_t s) {
  // Two rows a warp share the tokens' reads and conversions, which count from
  // four tokens on; one when two would leave too few blocks: two an SM for the
  // weights' loads (l = 1 at 4096 -> 4096: 8.5 us with one row, 10.1 with two),
  // one for the conversions (l = 8: 31 and 22).  What registers are left hold strips in flight.
  const int64_t two = static_cast<int64_t>((L <= 2 ? 4 : 2) * kSkWarps) * sm_count();
  return a.N >= two ? skinny_t<L, 2, L <= 2 ? 2 : 1>(a, s) : skinny_t<L, 1, L <= 4 ? 4 : 2>(a, s);
}

cudaError_t launch_fp8_skinny(const Fp8SkinnyArgs& a, cudaStream_t s) {
  switch (skinny_tokens(a.l)) {
    case 1: return skinny_l<1>(a, s);
    case 2: return skinny_l<2>(a, s);
    case 4: return skinny_l<4>(a, s);
    default: return skinny_l<8>(a, s);
  }
}

}  // namespace avr
