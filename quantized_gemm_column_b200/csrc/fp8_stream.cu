// Product of the experts' 8-bit rows with their weights when an expert has few
// rows (decoding): the weights are read once and that is what bounds it.
//   Y[r, f] = sum_b 2^(ea[r, b] + ew[f, b]) sum_{k in b} qa[r, k] qw[f, k]
//
// The kernel for many rows (fp8_gemm.cu) puts rows on the instruction's M side,
// 256 of them, so a pair that has 2 rows of an expert computes 256, and its
// stages carry 16 KB of rows beside 16 KB of weights.  Here the weights are the
// M side: a CTA pair takes 256 features of an expert and one 128-row block of
// its tokens, N of them (the tokens there are, rounded up to 32).  Each CTA
// loads 128 rows of weights (16 KB a stage) and half of the tokens' rows (8 KB
// at most), so eight stages fit and an SM keeps 128 KB of weights in flight;
// the MMAs of a stage take a third of the time its weights need from HBM.
// The accumulator is transposed, features in tensor memory's lanes and tokens
// in its columns: a warp writes 32 consecutive features of a token at a time.
//
// Roles as in fp8_gemm.cu: eight epilogue warps, an MMA thread and a scale
// copier in the leading CTA, TMA producers of weights (two), of tokens and of scales.
#include "fp8_pair.cuh"

namespace avr {

using namespace pair;
using namespace fp8;

namespace {

struct StreamCfg {
  static constexpr int kBM = 128;                               // features of a CTA (256 of a pair)
  static constexpr int kMaxN = 128;                             // tokens of a tile
  static constexpr int kBoxRows = 16;                           // tokens of a copy: N / 2 is a multiple
  static constexpr int kStages = 8;                             // 128 of K each
  static constexpr int kABytes = kBM * 128, kBBytes = kMaxN / 2 * 128;
  static constexpr int kSlots = 2;                              // scale atoms: 512 of K each
  static constexpr int kSfBytes = 512;                          // one atom of weights, one of tokens
  static constexpr int kEpiWarps = 8;                           // warps 0..7: warp % 4 is the lane quarter
  static constexpr int kMmaWarp = 8, kWeightWarp = 9, kTokenWarp = 11, kScaleWarp = 12, kCopyWarp = 13;
  static constexpr int kThreads = 512;                          // as many as the counts' scan takes
  static constexpr int kSfaOffset = kStages * (kABytes + kBBytes);
  static constexpr int kSfbOffset = kSfaOffset + kSlots * kSfBytes;
  static constexpr int kBarOffset = kSfbOffset + kSlots * kSfBytes;
  static constexpr int kBufferOffset = kBarOffset + 256;
  static constexpr int kSmemBytes = kBufferOffset + static_cast<int>(sizeof(Buffer));
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  // tensor memory: two accumulators, then the scale slots
  static constexpr int kSfaCol = 2 * kMaxN, kSfbCol = kSfaCol + 4 * kSlots;
  static constexpr int kTmemCols = 512;
  // instruction descriptor: E4M3 A and B (0), E8M0 scales (bit 23), K-major,
  // M >> 4 at bit 24; N >> 3 at bit 17 and the scale bytes at bits 4 and 29 are a tile's and a block's
  static constexpr uint32_t kIdesc = (1u << 23) | (static_cast<uint32_t>((2 * kBM) >> 4) << 24);
};

struct StreamParams {
  int64_t N, l_cap;
  int E, tiles_n, nkb;
  const int32_t* counts;
  void* Y;
  uint32_t* status;
};

struct StreamTile {
  int32_t f0;          // first feature of the pair's 256, in the expert
  int32_t w_row;       // this CTA's first row of the stacked weights
  int32_t row0, rows;  // the block's first row, its tokens
  int32_t n;           // tokens rounded up to 32
};

__device__ __forceinline__ StreamTile stream_tile(const StreamParams& p, const Buffer* b, int i, int rank) {
  // features fastest: the pairs working at one time read one expert's tokens and all of its weights
  const int mt = i / p.tiles_n, e = expert_of_tile(b, p.E, mt);
  const int off = 128 * (mt - (e > 0 ? b->tile_end[e - 1] : 0));
  StreamTile t;
  t.f0 = i % p.tiles_n * 256;
  t.w_row = e * static_cast<int32_t>(p.N) + t.f0 + rank * 128;
  t.row0 = 128 * (e > 0 ? b->blk_end[e - 1] : 0) + off;
  t.rows = min(128, b->rows[e] - off);
  t.n = (t.rows + 31) / 32 * 32;
  return t;
}

}  // namespace

template <bool kBf16Out>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(StreamCfg::kThreads, 1)
    fp8_stream_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_sfw, const __grid_constant__ CUtensorMap map_sfx,
                      const StreamParams p) {
  using Cfg = StreamCfg;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the swizzled tiles need 1024-byte alignment; a CTA without it still takes
  // part in the pair's cluster barriers and allocation, but does no work
  const bool aligned = (smem_u32(smem_raw) & 1023u) == 0;
  uint8_t* sA = smem_raw;
  uint8_t* sB = sA + Cfg::kStages * Cfg::kABytes;
  uint8_t* sSfa = smem_raw + Cfg::kSfaOffset;
  uint8_t* sSfb = smem_raw + Cfg::kSfbOffset;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw + Cfg::kBarOffset);   // [kStages] leading CTA
  uint64_t* empty = full + Cfg::kStages;        // [kStages] both CTAs
  uint64_t* sf_full = empty + Cfg::kStages;     // [kSlots] leading CTA
  uint64_t* sf_empty = sf_full + Cfg::kSlots;   // [kSlots] both CTAs
  uint64_t* sf_ready = sf_empty + Cfg::kSlots;  // [kSlots] leading CTA: in tensor memory
  uint64_t* acc_full = sf_ready + Cfg::kSlots;  // [2] both CTAs
  uint64_t* acc_empty = acc_full + 2;           // [2] leading CTA: every epilogue warp of both
  uint64_t* drained = acc_empty + 2;            // [2] leading CTA: the MMA and copy threads'
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);
  Buffer* buffer = reinterpret_cast<Buffer*>(smem_raw + Cfg::kBufferOffset);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool lead = rank == 0;

  if (threadIdx.x == 0) {
    if (!aligned) raise_status(p.status, AVR_ERR_MISALIGNED);
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
    prefetch_tensormap(&map_sfw);
    prefetch_tensormap(&map_sfx);
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full[s], 2);                   // the leading CTA's producers of weights and of tokens
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < Cfg::kSlots; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], 1);
      mbar_init(&sf_ready[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 2 * Cfg::kEpiWarps);
      mbar_init(&drained[a], 1);
    }
    fence_mbarrier_init();
  }
  if (warp == Cfg::kMmaWarp) {
    tmem_alloc_pair(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();          // barriers initialised and tensor memory allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();

  const int pairs = static_cast<int>(gridDim.x) / 2, pair = static_cast<int>(blockIdx.x) / 2;
  int num_tiles = scan_counts<Cfg::kThreads, 1>(p.counts, p.E, p.l_cap, buffer, p.status) * p.tiles_n;
  // both CTAs of a pair, of one launch, are aligned or neither is
  if (!aligned) num_tiles = 0;
  auto tile = [&](int i) { return stream_tile(p, buffer, i, rank); };

  if (warp >= Cfg::kWeightWarp && warp <= Cfg::kTokenWarp) {
    if (elect_one()) {
      // ---------------- weights (two threads, alternate stages) and tokens ----------------
      const bool weights = warp < Cfg::kTokenWarp;
      const int parity = warp - Cfg::kWeightWarp;
      const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
      int it = 0;
      bool ok = true;
      for (int i = pair; i < num_tiles && ok; i += pairs) {
        const StreamTile t = tile(i);
        for (int kb = 0; kb < p.nkb; ++kb, ++it) {
          if (weights && (it & 1) != parity) continue;
          const int st = it % Cfg::kStages;
          const uint32_t ph = static_cast<uint32_t>(it / Cfg::kStages) & 1u;
          if (it >= Cfg::kStages && !mbar_wait_backoff(&empty[st], ph ^ 1u, p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = full_lead + static_cast<uint32_t>(st * 8);
          const int half = t.n / 2;             // the instruction takes half of its N tokens from each CTA
          if (lead) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(2 * (weights ? Cfg::kABytes : 128 * half)));
          if (weights)
            tma_load_2d_pair(sA + st * Cfg::kABytes, &map_w, bar, 128 * kb, t.w_row);
          else
            for (int r = 0; r < half; r += Cfg::kBoxRows)
              tma_load_2d_pair(sB + st * Cfg::kBBytes + 128 * r, &map_x, bar, 128 * kb, t.row0 + rank * half + r);
        }
      }
    }
  } else if (warp == Cfg::kScaleWarp) {
    if (elect_one()) {
      // ---------------- scale producer: the atoms of 512 of K ----------------
      const uint32_t bar_lead = mapa_shared(smem_u32(sf_full), 0);
      int it = 0;
      bool ok = true;
      for (int i = pair; i < num_tiles && ok; i += pairs) {
        const StreamTile t = tile(i);
        for (int c = 0; c <= (p.nkb - 1) >> 2; ++c, ++it) {
          const int sl = it % Cfg::kSlots;
          const uint32_t ph = static_cast<uint32_t>(it / Cfg::kSlots) & 1u;
          if (it >= Cfg::kSlots && !mbar_wait_backoff(&sf_empty[sl], ph ^ 1u, p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = bar_lead + static_cast<uint32_t>(sl * 8);
          if (lead) mbar_arrive_expect_tx(&sf_full[sl], 2 * 2 * Cfg::kSfBytes);
          tma_load_2d_pair(sSfa + sl * Cfg::kSfBytes, &map_sfw, bar, 64 * c, t.w_row >> 7);
          tma_load_2d_pair(sSfb + sl * Cfg::kSfBytes, &map_sfx, bar, 64 * c, t.row0 >> 7);
        }
      }
    }
  } else if (warp == Cfg::kCopyWarp) {
    if (lead && elect_one()) {
      // ---------------- scale copier (leading CTA; each copy fills both CTAs) ----------------
      // A slot's tensor-memory columns are free when its shared memory is: the
      // producer refilled it after the MMAs that read both had completed.
      int it = 0;
      bool ok = true;
      for (int i = pair; i < num_tiles && ok; i += pairs) {
        for (int c = 0; c <= (p.nkb - 1) >> 2; ++c, ++it) {
          const int sl = it % Cfg::kSlots;
          if (!mbar_wait_poll(&sf_full[sl], static_cast<uint32_t>(it / Cfg::kSlots) & 1u, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          tc_cp_32x128b_warpx4_pair(tmem + Cfg::kSfaCol + 4 * sl,
                                    smem_desc(smem_u32(sSfa + sl * Cfg::kSfBytes), 0, 128, kLayoutSwizzleNone));
          tc_cp_32x128b_warpx4_pair(tmem + Cfg::kSfbCol + 4 * sl,
                                    smem_desc(smem_u32(sSfb + sl * Cfg::kSfBytes), 0, 128, kLayoutSwizzleNone));
          tc_commit_pair(&sf_ready[sl]);
        }
      }
      tc_commit_pair(&drained[1]);
      mbar_wait(&drained[1], 0, p.status);
    }
  } else if (warp == Cfg::kMmaWarp) {
    if (lead && elect_one()) {
      // ---------------- MMA issuer (leading CTA) ----------------
      int st = 0, sl = 0, done = 0;
      uint32_t ph = 0, sph = 0;
      bool ok = true;
      for (int i = pair; i < num_tiles && ok; i += pairs, ++done) {
        const int acc = done & 1;
        const uint32_t d = tmem + static_cast<uint32_t>(Cfg::kMaxN * acc);
        const uint32_t idesc_n = Cfg::kIdesc | (static_cast<uint32_t>(tile(i).n >> 3) << 17);
        if (done >= 2 && !mbar_wait_poll(&acc_empty[acc], static_cast<uint32_t>(done / 2 - 1) & 1u, p.status)) break;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if ((kb & 3) == 0 && !mbar_wait_poll(&sf_ready[sl], sph, p.status)) {
            ok = false;
            break;
          }
          if (!mbar_wait_poll(&full[st], ph, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a0 = smem_desc(smem_u32(sA + st * Cfg::kABytes), 16, 1024, kLayoutSwizzle128B);
          const uint64_t b0 = smem_desc(smem_u32(sB + st * Cfg::kBBytes), 16, 1024, kLayoutSwizzle128B);
          const uint32_t byte = static_cast<uint32_t>(kb & 3);
          const uint32_t idesc = idesc_n | (byte << 4) | (byte << 29);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mma_fp8_pair(d, a0 + static_cast<uint64_t>(2 * q), b0 + static_cast<uint64_t>(2 * q), idesc,
                         tmem + Cfg::kSfaCol + 4 * sl, tmem + Cfg::kSfbCol + 4 * sl, (kb > 0 || q > 0) ? 1u : 0u);
          tc_commit_pair_both(&empty[st]);
          if ((kb & 3) == 3 || kb + 1 == p.nkb) {
            tc_commit_pair_both(&sf_empty[sl]);
            if (++sl == Cfg::kSlots) {
              sl = 0;
              sph ^= 1u;
            }
          }
          if (++st == Cfg::kStages) {
            st = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair_both(&acc_full[acc]);
      }
      tc_commit_pair(&drained[0]);
      mbar_wait(&drained[0], 0, p.status);
    }
  } else if (warp < Cfg::kEpiWarps) {
    // ---------------- epilogue (both CTAs, own features) ----------------
    const int q = warp & 3, h = warp / 4;       // lane quarter of tensor memory; which 64 tokens
    const uint32_t acc_empty_lead = mapa_shared(smem_u32(acc_empty), 0);
    int done = 0;
    for (int i = pair; i < num_tiles; i += pairs, ++done) {
      const StreamTile t = tile(i);
      const int acc = done & 1;
      uint32_t okw = 0;
      if (lane == 0) okw = mbar_wait_backoff(&acc_full[acc], static_cast<uint32_t>(done / 2) & 1u, p.status) ? 1u : 0u;
      if (__shfl_sync(0xFFFFFFFFu, okw, 0) == 0u) break;
      tc_fence_after();
      const uint32_t t_row = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(Cfg::kMaxN * acc);
      const int64_t f = t.f0 + rank * 128 + 32 * q + lane;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n0 = 64 * h + 32 * c;
        if (n0 >= t.rows) break;                // the whole warp
        uint32_t v[32];
        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(n0), v);
        tmem_ld_wait();
        if (f >= p.N) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if (n0 + k >= t.rows) break;
          const int64_t at = (static_cast<int64_t>(t.row0) + n0 + k) * p.N + f;
          if (kBf16Out)
            static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(__uint_as_float(v[k]));
          else
            static_cast<float*>(p.Y)[at] = __uint_as_float(v[k]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty_lead + static_cast<uint32_t>(8 * acc));
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();          // no CTA leaves while its pair may still signal its barriers
  if (warp == Cfg::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, Cfg::kTmemCols);
  }
}

// For a buffer of up to two 128-row blocks an expert (the counts are the
// device's); us here / with the rows first, 64 experts of 2048 -> 1024, top 8:
//   16 tokens  15.2 / 18.3    256 tokens  28.0 / 29.6    1000 tokens  38.2 / 40.0
// (reading the experts' weights takes 9.9, 17.2 and 18.8).  Above, a block of
// rows at a time reads the weights too often.  fp32 sums longer than a visit of
// fp8_gemm.cu's go there.
bool fp8_stream_applies(const Fp8GemmArgs& a) {
  return a.mode == Fp8GemmArgs::kRows && a.a_rows <= 128 * static_cast<int64_t>(a.E) * kStreamBlocks &&
         (a.yt == AVR_BF16 || blocks128(a.K) <= kFp8MaxVisit);
}

template <bool kBf16Out>
static cudaError_t stream_t(const Fp8GemmArgs& a, cudaStream_t s) {
  using Cfg = StreamCfg;
  CUtensorMap mw, mx, msw, msx;
  const uint64_t K = static_cast<uint64_t>(a.K), sf_cols = static_cast<uint64_t>(atoms128(a.K)) * 64;
  if (!make_tensor_map_2d(&mw, a.b_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, static_cast<uint64_t>(a.b_rows), K,
                          Cfg::kBM, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_2d(&mx, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, static_cast<uint64_t>(a.a_rows), K,
                          Cfg::kBoxRows, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_2d(&msw, a.b_scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8,
                          static_cast<uint64_t>(blocks128(a.b_rows)), sf_cols, 1, 64, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tensor_map_2d(&msx, a.a_scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8,
                          static_cast<uint64_t>(blocks128(a.a_rows)), sf_cols, 1, 64, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  StreamParams p = {};
  p.N = a.N;
  p.l_cap = a.a_rows;
  p.E = a.E;
  p.tiles_n = static_cast<int>((a.N + 255) / 256);
  p.nkb = static_cast<int>(blocks128(a.K));
  p.counts = a.counts;
  p.Y = a.Y;
  p.status = a.status;
  const int64_t tiles = a.a_rows / 128 * p.tiles_n;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto kern = fp8_stream_kernel<kBf16Out>;
  const void* fn = reinterpret_cast<const void*>(kern);
  cudaError_t e = set_max_dynamic_smem(fn, Cfg::kSmemBytes);
  if (e != cudaSuccess) return e;
  static std::atomic<int> resident[kFp8CachedDevices];
  const int most = fp8_resident_pairs(fn, Cfg::kThreads, Cfg::kSmemBytes, resident);
  const int pairs = static_cast<int>(tiles < most ? tiles : most);
  return launch_ex(kern, dim3(2 * pairs), dim3(Cfg::kThreads), Cfg::kSmemBytes, s, true, mw, mx, msw, msx, p);
}

cudaError_t launch_fp8_stream(const Fp8GemmArgs& a, cudaStream_t s) {
  return a.yt == AVR_BF16 ? stream_t<true>(a, s) : stream_t<false>(a, s);
}

}  // namespace avr
