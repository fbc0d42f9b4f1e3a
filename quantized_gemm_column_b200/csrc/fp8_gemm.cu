// Product of two E4M3 tensors with a power-of-two scale per block of 128, on
// the 5th-generation tensor cores:
//   Y[i, j] = sum_b 2^(ea[i, b] + eb[j, b]) sum_{k in b} qa[i, k] qb[j, k].
// The scales are exponents (E8M0), so tcgen05.mma.kind::mxf8f6f4.block_scale
// applies them inside the tensor core and the fp32 accumulator never leaves
// tensor memory until a tile is done.
//
// The instruction scales 32 elements at a time; a block of 128 is four
// instructions that read the same byte.  A scale word in tensor memory has
// four bytes and the instruction descriptor picks one, so a 512-byte atom
// (128 rows x 4 blocks) serves 512 of K: three copies of scales (one of A's
// atoms, two of B's) per 16 MMAs.
//
// Persistent CTA pairs (cta_group::2) on 256 x 256 tiles, as the FP4 pair
// kernel: each CTA holds its 128 rows of A and half of B, so an SM loads 32 KB
// for the 2 * 128 * 256 * 128 flop of its share of a stage.
//   warp 0      : tensor-memory allocation; in the leading CTA one thread
//                 issues the pair's MMAs;
//   warps 1..4  : TMA producers of A and B, two each, alternate stages;
//   warp 5      : producer of the scale atoms, two slots of 512 of K;
//   warp 6      : in the leading CTA one thread copies the scales into tensor
//                 memory, a slot ahead of the MMAs, which would wait for
//                 copies of their own thread;
//   warps 8..15 : epilogue, each a lane quarter of one 128-column half, through
//                 a 4 KB staging box of its own and a TMA store.
//
// Accumulators.  Two tiles' 512 columns would fill tensor memory and leave
// nothing for scales, so consecutive tiles start at columns 0 and 224 and
// share 32 columns.  The epilogue takes a tile's shared columns out first and
// then lets the next tile's MMAs start, so the rest of the drain, the
// conversion and the stores run under them.
//
// The tensor core's fp32 sums are cut off, not rounded, so a long sum of one
// sign drifts (1e-6 relative over 4096 terms, 9e-6 over 16384).  An fp32
// output is therefore summed in visits of at most 6144 of K: the first is
// stored, the others are added to it by TMA reductions, which round to nearest,
// in order.  A bf16 output is one sum: its own rounding is 400 times the drift
// of 16384 terms; 2^20 terms of one sign can be cut off by as much.
//
// When the last round of an fp32 output has tiles for less than half of the
// pairs, each of them is cut along K among several pairs (parts).  A part adds
// to what the part below it has stored: it waits for a pair of lower index,
// which the hardware starts no later, in the same round.  So the order of the
// additions, and the bits, are fixed.
//
// Three uses, one code path: one product; the experts' buffer by row tiles
// (kRows: a tile's rows belong to one expert, whose B is stacked); the
// experts' weight gradients (kTokens: one product per expert, K = its tokens,
// whose blocks may start at any byte of an atom).
#include "fp8_pair.cuh"

namespace avr {

using namespace pair;
using namespace fp8;

namespace {

constexpr int kMinPart = 12;

struct Cfg {
  static constexpr int kBM = 128, kBN = 256, kBNHalf = 128;     // per CTA; a pair's tile is 256 x 256
  static constexpr int kStages = 5;                             // 128 of K each
  static constexpr int kABytes = kBM * 128, kBBytes = kBNHalf * 128;
  static constexpr int kSlots = 2;                              // scale atoms: 512 of K each
  static constexpr int kSfaBytes = 512, kSfbBytes = 1024;
  static constexpr int kProducers = 4;
  static constexpr int kScaleWarp = 1 + kProducers;
  static constexpr int kCopyWarp = kScaleWarp + 1;
  static constexpr int kFirstEpiWarp = 8, kEpiWarps = 8;
  static constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
  static constexpr int kBoxBytes = 32 * 128;                    // an epilogue warp's staging box
  static constexpr int kOutOffset = kStages * (kABytes + kBBytes);
  static constexpr int kSfaOffset = kOutOffset + kEpiWarps * kBoxBytes;
  static constexpr int kSfbOffset = kSfaOffset + kSlots * kSfaBytes;
  static constexpr int kBarOffset = kSfbOffset + kSlots * kSfbBytes;
  static constexpr int kSmemBytes = kBarOffset + 256;
  static_assert(kSmemBytes + 3 * 4 * kMaxExperts + 256 <= 227 * 1024, "shared memory budget");
  // tensor memory: the accumulators at columns 0 and 224, then the scale slots
  static constexpr int kAccStep = 224;
  static constexpr int kSfaCol = kAccStep + kBN;                // 480
  static constexpr int kSfbCol = kSfaCol + 4 * kSlots;
  static constexpr int kTmemCols = 512;
  static_assert(kSfbCol + 8 * kSlots <= kTmemCols, "tensor memory budget");
  // instruction descriptor: E4M3 A and B (0), E8M0 scales (bit 23), K-major,
  // N >> 3 at bit 17, M >> 4 at bit 24; the scale byte of B at bit 4, of A at 29
  static constexpr uint32_t kIdesc = (static_cast<uint32_t>(kBN >> 3) << 17) | (1u << 23) |
                                     (static_cast<uint32_t>((2 * kBM) >> 4) << 24);
};

struct Params {
  int64_t M, N;
  int tiles_m, tiles_n, nkb;      // kTokens: per expert, nkb unused
  int num_tiles;                  // kRows: at most; the counts give the rest
  int cut0, parts;                // tiles from cut0 on are cut into parts (kDense, fp32; else past the end, 1)
  int a_oob;                      // a row coordinate past A: reads zeros
  int y_passes;                   // Y is larger than L2 holds: it goes first, the operands stay
  int E;
  const int32_t* counts;          // kRows: the experts' tokens, turned into row tiles by every CTA
  Fp8Table t;                     // kTokens
  void* Y;
  uint32_t* flags;                // [pairs][2][8], zero between launches: a warp's share of a part is stored
  uint32_t* status;
};

// what one CTA of the pair does for a tile
struct Tile {
  int32_t a_row, b_row;           // first operand rows (b_row: of this CTA's half)
  int32_t b_row0;                 // first B row of the whole tile (scales)
  int32_t n0, kb0, nkb;
  int64_t y_row;
  int32_t rows;                   // rows of this CTA's 128 to be stored (<= 0: none)
  int32_t part;                   // kDense: which part of the tile (0: all, or the first)
};

template <int kMode>
__device__ __forceinline__ Tile tile_at(const Params& p, const Buffer* b, int i, int rank) {
  Tile t;
  t.part = 0;
  if (kMode == Fp8GemmArgs::kDense) {
    t.kb0 = 0;
    t.nkb = p.nkb;
    if (i >= p.cut0) {
      const int item = i - p.cut0;
      i = p.cut0 + item / p.parts;
      t.part = item % p.parts;
      t.kb0 = p.nkb * t.part / p.parts;
      t.nkb = p.nkb * (t.part + 1) / p.parts - t.kb0;
    }
    // bands of 8 column tiles, rows outside, so that the pairs working at one
    // time share both operands' tiles in L2
    const int band = i / (8 * p.tiles_m), r = i - band * 8 * p.tiles_m;
    const int width = min(8, p.tiles_n - 8 * band);
    const int m0 = r / width * 256 + rank * 128;
    t.n0 = (8 * band + r % width) * 256;
    t.a_row = m0;
    t.b_row0 = t.n0;
    t.y_row = m0;
    t.rows = static_cast<int32_t>(min64(128, p.M - m0));
  } else if (kMode == Fp8GemmArgs::kRows) {
    const int mt = i / p.tiles_n, lo = expert_of_tile(b, p.E, mt);
    const int off = 256 * (mt - (lo > 0 ? b->tile_end[lo - 1] : 0));
    const int row0 = 128 * (lo > 0 ? b->blk_end[lo - 1] : 0) + off + rank * 128;
    t.n0 = i % p.tiles_n * 256;
    t.rows = min(128, b->rows[lo] - off - rank * 128);
    t.a_row = t.rows > 0 ? row0 : p.a_oob;               // the other CTA's block may be another expert's
    t.b_row0 = lo * static_cast<int32_t>(p.N) + t.n0;
    t.kb0 = 0;
    t.nkb = p.nkb;
    t.y_row = row0;
  } else {
    // The experts come with the most tokens first and every other round of
    // tiles goes to the pairs backwards, so that the pairs' sums of blocks come
    // out alike (in the experts' own order a few large ones decide the time).
    const int per = p.tiles_m * p.tiles_n, pairs = static_cast<int>(gridDim.x) / 2, round = i / pairs;
    if ((round & 1) != 0 && (round + 1) * pairs <= p.num_tiles) i = (2 * round + 1) * pairs - 1 - i;
    const int r = i % per, e = __ldcg(p.t.order + i / per);
    const int2 sg = __ldcg(reinterpret_cast<const int2*>(p.t.seg) + e);
    const int m0 = r / p.tiles_n * 256 + rank * 128;
    t.n0 = r % p.tiles_n * 256;
    t.rows = static_cast<int32_t>(min64(128, p.M - m0));
    t.a_row = m0;
    t.b_row0 = t.n0;
    t.kb0 = sg.x >> 7;
    t.nkb = (sg.y + 127) >> 7;
    t.y_row = e * p.M + m0;
  }
  t.b_row = t.b_row0 + rank * 128;
  return t;
}

// blocks of K in a visit of a tile of n: n, or the fewest equal visits for fp32
template <bool kBf16Out>
__device__ __forceinline__ int visit_length(int n) {
  const int visits = (n + kFp8MaxVisit - 1) / kFp8MaxVisit;
  return kBf16Out || visits < 2 ? n : (n + visits - 1) / visits;
}

// TMA store shared -> global under an L2 policy
__device__ __forceinline__ void tma_store_2d_policy(const CUtensorMap* map, const void* src, int32_t x, int32_t y,
                                                    uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3}], [%1], %4;"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(x), "r"(y), "l"(policy)
               : "memory");
}

// TMA reduction shared -> global: adds, each element rounded to nearest
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int32_t x, int32_t y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}

// a flag that a thread sets after its stores completed, and one of another CTA
// waits for, as long as the workspace's bound says, and hands back
__device__ __forceinline__ void flag_set(uint32_t* f) {
  fence_proxy_async_global();
  __threadfence();
  asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(f) : "memory");
}
__device__ __forceinline__ bool flag_take(uint32_t* f, uint32_t* status) {
  const uint64_t t0 = globaltimer_ns();
  uint64_t limit = 0;
  for (;;) {
    uint32_t x;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(f) : "memory");
    if (x != 0u) break;
    if (limit == 0) {                 // the status word is the workspace's first
      limit = __ldcg(reinterpret_cast<const uint64_t*>(reinterpret_cast<const char*>(status) + kWaitLimitOffset));
      if (limit == 0) limit = kWaitLimitNs;
    }
    if (globaltimer_ns() - t0 > limit) {
      raise_status(status, AVR_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
  *f = 0u;
  fence_proxy_async_global();
  return true;
}

}  // namespace

template <int kMode, bool kBf16Out>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg::kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_sfa, const __grid_constant__ CUtensorMap map_sfb,
                    const __grid_constant__ CUtensorMap map_y, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the swizzled tiles need 1024-byte alignment; a CTA without it still takes
  // part in the pair's cluster barriers and allocation, but does no work
  const bool aligned = (smem_u32(smem_raw) & 1023u) == 0;
  uint8_t* sA = smem_raw;
  uint8_t* sB = sA + Cfg::kStages * Cfg::kABytes;
  uint8_t* sOut = smem_raw + Cfg::kOutOffset;
  uint8_t* sSfa = smem_raw + Cfg::kSfaOffset;
  uint8_t* sSfb = smem_raw + Cfg::kSfbOffset;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw + Cfg::kBarOffset);   // [kStages] leading CTA: A, B landed
  uint64_t* empty = full + Cfg::kStages;        // [kStages] both CTAs
  uint64_t* sf_full = empty + Cfg::kStages;     // [kSlots] leading CTA: scale atoms landed in both CTAs
  uint64_t* sf_empty = sf_full + Cfg::kSlots;   // [kSlots] both CTAs
  uint64_t* sf_ready = sf_empty + Cfg::kSlots;  // [kSlots] leading CTA: in tensor memory
  uint64_t* acc_full = sf_ready + Cfg::kSlots;  // both CTAs
  uint64_t* acc_empty = acc_full + 1;           // leading CTA: every epilogue warp of both
  uint64_t* drained = acc_empty + 1;            // [2] leading CTA: the MMA and copy threads'
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool lead = rank == 0;

  if (threadIdx.x == 0) {
    if (!aligned) raise_status(p.status, AVR_ERR_MISALIGNED);
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    prefetch_tensormap(&map_sfa);
    prefetch_tensormap(&map_sfb);
    prefetch_tensormap(&map_y);
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&full[s], 2);                   // the leading CTA's A and B producers
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < Cfg::kSlots; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], 1);
      mbar_init(&sf_ready[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * Cfg::kEpiWarps);
    mbar_init(&drained[0], 1);
    mbar_init(&drained[1], 1);
    fence_mbarrier_init();
  }
  if (warp == 0) {
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
  int num_tiles = p.num_tiles;
  Buffer* buffer = reinterpret_cast<Buffer*>(smem_raw + Cfg::kSmemBytes);
  if (kMode == Fp8GemmArgs::kRows) num_tiles = scan_counts<Cfg::kThreads, 2>(p.counts, p.E, p.M, buffer, p.status) * p.tiles_n;
  if (kMode == Fp8GemmArgs::kTokens && __ldcg(p.t.fits) == 0) num_tiles = 0;   // the counts did not fit
  // both CTAs of a pair leave their loops together: a CTA whose shared memory
  // is misaligned has a misaligned partner (same launch), so neither works
  if (!aligned) num_tiles = 0;

  if (warp >= 1 && warp <= Cfg::kProducers) {
    if (elect_one()) {
      // ---------------- A and B producers ----------------
      const bool is_a = warp <= 2;
      const int parity = (warp - 1) & 1;
      const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
      int it = 0;
      bool ok = true;
      for (int i = pair; i < num_tiles && ok; i += pairs) {
        const Tile t = tile_at<kMode>(p, buffer, i, rank);
        for (int kb = t.kb0; kb < t.kb0 + t.nkb; ++kb, ++it) {
          if ((it & 1) != parity) continue;
          const int st = it % Cfg::kStages;
          const uint32_t ph = static_cast<uint32_t>(it / Cfg::kStages) & 1u;
          if (it >= Cfg::kStages && !mbar_wait_backoff(&empty[st], ph ^ 1u, p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = full_lead + static_cast<uint32_t>(st * 8);
          if (lead) mbar_arrive_expect_tx(&full[st], 2 * (is_a ? Cfg::kABytes : Cfg::kBBytes));
          if (is_a)
            tma_load_2d_pair(sA + st * Cfg::kABytes, &map_a, bar, 128 * kb, t.a_row);
          else
            tma_load_2d_pair(sB + st * Cfg::kBBytes, &map_b, bar, 128 * kb, t.b_row);
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
        const Tile t = tile_at<kMode>(p, buffer, i, rank);
        if (t.nkb == 0) continue;
        for (int c = t.kb0 >> 2; c <= (t.kb0 + t.nkb - 1) >> 2; ++c, ++it) {
          const int sl = it % Cfg::kSlots;
          const uint32_t ph = static_cast<uint32_t>(it / Cfg::kSlots) & 1u;
          if (it >= Cfg::kSlots && !mbar_wait(&sf_empty[sl], ph ^ 1u, p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = bar_lead + static_cast<uint32_t>(sl * 8);
          if (lead) mbar_arrive_expect_tx(&sf_full[sl], 2 * (Cfg::kSfaBytes + Cfg::kSfbBytes));
          tma_load_2d_pair(sSfa + sl * Cfg::kSfaBytes, &map_sfa, bar, 64 * c, t.a_row >> 7);
          tma_load_2d_pair(sSfb + sl * Cfg::kSfbBytes, &map_sfb, bar, 64 * c, t.b_row0 >> 7);
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
        const Tile t = tile_at<kMode>(p, buffer, i, 0);
        if (t.nkb == 0) continue;
        for (int c = t.kb0 >> 2; c <= (t.kb0 + t.nkb - 1) >> 2; ++c, ++it) {
          const int sl = it % Cfg::kSlots;
          if (!mbar_wait_poll(&sf_full[sl], static_cast<uint32_t>(it / Cfg::kSlots) & 1u, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = smem_desc(smem_u32(sSfa + sl * Cfg::kSfaBytes), 0, 128, kLayoutSwizzleNone);
          const uint64_t db = smem_desc(smem_u32(sSfb + sl * Cfg::kSfbBytes), 0, 128, kLayoutSwizzleNone);
          const uint32_t sfb_t = tmem + Cfg::kSfbCol + 8 * sl;
          tc_cp_32x128b_warpx4_pair(tmem + Cfg::kSfaCol + 4 * sl, da);
          tc_cp_32x128b_warpx4_pair(sfb_t, db);
          tc_cp_32x128b_warpx4_pair(sfb_t + 4, db + 32);
          tc_commit_pair(&sf_ready[sl]);
        }
      }
      tc_commit_pair(&drained[1]);
      mbar_wait(&drained[1], 0, p.status);
    }
  } else if (warp == 0) {
    if (lead && elect_one()) {
      // ---------------- MMA issuer (leading CTA) ----------------
      int st = 0, sl = 0, done = 0;
      uint32_t ph = 0, sph = 0;
      bool ok = true;
      for (int i = pair; i < num_tiles && ok; i += pairs) {
        const Tile t = tile_at<kMode>(p, buffer, i, 0);
        if (t.nkb == 0) continue;
        uint32_t d = tmem + static_cast<uint32_t>(Cfg::kAccStep * (done & 1));
        const int end = t.kb0 + t.nkb;
        const int visit = visit_length<kBf16Out>(t.nkb);
        int kb0 = t.kb0;                        // the visit's first block
        for (int kb = t.kb0; kb < end; ++kb) {
          if (!kBf16Out && kb == kb0 + visit) {
            tc_commit_pair_both(acc_full);
            ++done;
            d = tmem + static_cast<uint32_t>(Cfg::kAccStep * (done & 1));
            kb0 = kb;
          }
          const uint32_t sfa_t = tmem + Cfg::kSfaCol + 4 * sl, sfb_t = tmem + Cfg::kSfbCol + 8 * sl;
          if (kb == t.kb0 || (kb & 3) == 0) {
            if (!mbar_wait_poll(&sf_ready[sl], sph, p.status)) {
              ok = false;
              break;
            }
          }
          if (!mbar_wait_poll(&full[st], ph, p.status) ||
              (kb == kb0 && done >= 1 &&
               !mbar_wait_poll(acc_empty, static_cast<uint32_t>(done - 1) & 1u, p.status))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a0 = smem_desc(smem_u32(sA + st * Cfg::kABytes), 16, 1024, kLayoutSwizzle128B);
          const uint64_t b0 = smem_desc(smem_u32(sB + st * Cfg::kBBytes), 16, 1024, kLayoutSwizzle128B);
          const uint32_t byte = static_cast<uint32_t>(kb & 3);
          const uint32_t idesc = Cfg::kIdesc | (byte << 4) | (byte << 29);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mma_fp8_pair(d, a0 + static_cast<uint64_t>(2 * q), b0 + static_cast<uint64_t>(2 * q), idesc, sfa_t, sfb_t,
                         (kb > kb0 || q > 0) ? 1u : 0u);
          tc_commit_pair_both(&empty[st]);
          if ((kb & 3) == 3 || kb + 1 == end) {
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
        tc_commit_pair_both(acc_full);
        ++done;
      }
      tc_commit_pair(&drained[0]);
      mbar_wait(&drained[0], 0, p.status);
    }
  } else if (warp >= Cfg::kFirstEpiWarp) {
    // ---------------- epilogue (both CTAs, own rows) ----------------
    const int q = warp & 3;                                // lane quarter of tensor memory this warp may read
    const int h = (warp - Cfg::kFirstEpiWarp) / 4;         // 128-column half
    uint8_t* box = sOut + (warp - Cfg::kFirstEpiWarp) * Cfg::kBoxBytes;
    const uint32_t acc_empty_lead = mapa_shared(smem_u32(acc_empty), 0);
    constexpr int kBoxCols = kBf16Out ? 64 : 32;           // 128 bytes of output
    constexpr int kBoxes = 128 / kBoxCols;
    constexpr int kElem = kBf16Out ? 2 : 4;
    uint64_t policy;
    if (p.y_passes)
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    else
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    // 32 output words of a box go out, w[k] at column col + k of row `lane`; add: to what is there
    auto store_box = [&](const uint32_t (&w)[32], int rows, int64_t y_row, int64_t col, bool add) {
      if (rows <= 0 || col >= p.N) return;                 // the whole warp
      if (kMode == Fp8GemmArgs::kRows && rows < 32) {
        // the last rows of a segment: the rows behind them are not written
        if (lane < rows) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.Y) + ((y_row + lane) * p.N + col) * kElem);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            if (col + u * (16 / kElem) >= p.N) continue;
            uint4 x = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
            if (!kBf16Out && add) {
              const uint4 y = dst[u];
              x = make_uint4(__float_as_uint(__uint_as_float(y.x) + __uint_as_float(x.x)),
                             __float_as_uint(__uint_as_float(y.y) + __uint_as_float(x.y)),
                             __float_as_uint(__uint_as_float(y.z) + __uint_as_float(x.z)),
                             __float_as_uint(__uint_as_float(y.w) + __uint_as_float(x.w)));
            }
            dst[u] = x;
          }
        }
        return;
      }
      if (lane == 0) bulk_wait_group_read<0>();            // the box's previous store has read it
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<uint4*>(box + lane * 128 + ((u ^ (lane & 7)) * 16)) =
            make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {                                     // clipped at Y's edges
        if (!kBf16Out && add)
          tma_add_2d(&map_y, box, static_cast<int32_t>(col), static_cast<int32_t>(y_row));
        else
          tma_store_2d_policy(&map_y, box, static_cast<int32_t>(col), static_cast<int32_t>(y_row), policy);
        bulk_commit_group();
      }
    };
    int done = 0;
    bool ok = true;
    for (int i = pair; i < num_tiles && ok; i += pairs) {
      const Tile t = tile_at<kMode>(p, buffer, i, rank);
      const int rows = t.rows - 32 * q;                    // of this warp's 32
      const int64_t y_row = t.y_row + 32 * q;
      if (t.nkb == 0) {                                    // an expert without tokens: a zero gradient
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = 0u;
        for (int bx = 0; bx < kBoxes; ++bx) store_box(w, rows, y_row, t.n0 + 128 * h + kBoxCols * bx, false);
        continue;
      }
      const bool cut = kMode == Fp8GemmArgs::kDense && !kBf16Out && i >= p.cut0;
      uint32_t* flag = p.flags + (static_cast<int64_t>(pair) * 2 + rank) * Cfg::kEpiWarps + (warp - Cfg::kFirstEpiWarp);
      const int visit = visit_length<kBf16Out>(t.nkb);
      for (int lo = 0; lo < t.nkb; lo += visit) {
        uint32_t okw = 1;
        if (lane == 0) {
          okw = mbar_wait_backoff(acc_full, static_cast<uint32_t>(done) & 1u, p.status) ? 1u : 0u;
          if (!kBf16Out) {
            if (lo > 0) bulk_wait_group_all();             // this tile's earlier visit is in memory
            // ... and so is the part below
            else if (cut && t.part > 0 && okw != 0) okw = flag_take(flag - 2 * Cfg::kEpiWarps, p.status) ? 1u : 0u;
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, okw, 0) != 0u;
        if (!ok) break;
        tc_fence_after();
        const bool odd = (done & 1) != 0;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(32 * q) << 16) +
                               static_cast<uint32_t>(Cfg::kAccStep * (odd ? 1 : 0) + 128 * h);
        // The columns shared with the next visit come out first: the last 32 of
        // an accumulator at column 0 (half 1), the first 32 of one at 224 (half
        // 0).  Every warp arrives once a visit, the visit before being done
        // with: then the next MMAs may write.
        bool owe = true;
        auto release = [&]() {
          if (owe) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_lead);
            owe = false;
          }
        };
        if (h != (odd ? 0 : 1)) release();
        for (int b = 0; b < kBoxes; ++b) {
          const int bx = odd ? b : kBoxes - 1 - b;
          uint32_t w[32];
          if (kBf16Out) {
            // 32 columns as 16 bf16 pairs
            auto load_pack = [&](int half) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(64 * bx + 32 * half), v);
              tmem_ld_wait();
              release();
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const __nv_bfloat162 pr = __floats2bfloat162_rn(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
                w[16 * half + k] = *reinterpret_cast<const uint32_t*>(&pr);
              }
            };
            if (odd) {
              load_pack(0);
              load_pack(1);
            } else {
              load_pack(1);
              load_pack(0);
            }
          } else {
            tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(32 * bx), w);
            tmem_ld_wait();
            release();
          }
          store_box(w, rows, y_row, t.n0 + 128 * h + kBoxCols * bx, lo > 0 || t.part > 0);
        }
        ++done;
      }
      if (cut && ok && t.part + 1 < p.parts && lane == 0) {
        bulk_wait_group_all();
        flag_set(flag);
      }
    }
    if (lane == 0) bulk_wait_group_all();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();          // no CTA leaves while its pair may still signal its barriers
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, Cfg::kTmemCols);
  }
}

int fp8_resident_pairs(const void* fn, int threads, size_t smem, std::atomic<int>* cache) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const bool kept = dev >= 0 && dev < kFp8CachedDevices;
  int n = kept ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (sm_count() / 2)));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) n = sm_count() / 2;
  if (kept) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int kMode, bool kBf16Out>
static cudaError_t gemm_t(const Fp8GemmArgs& a, cudaStream_t s) {
  CUtensorMap ma, mb, msa, msb, my;
  const uint64_t K = static_cast<uint64_t>(a.K), sf_cols = static_cast<uint64_t>(atoms128(a.K)) * 64;
  if (!make_tensor_map_2d(&ma, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, static_cast<uint64_t>(a.a_rows), K, 128, 128,
                          CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tensor_map_2d(&mb, a.b_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, static_cast<uint64_t>(a.b_rows), K, 128, 128,
                          CU_TENSOR_MAP_SWIZZLE_128B) ||
      // an atom as 64 eight-byte elements
      !make_tensor_map_2d(&msa, a.a_scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8,
                          static_cast<uint64_t>(blocks128(a.a_rows)), sf_cols, 1, 64, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tensor_map_2d(&msb, a.b_scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8,
                          static_cast<uint64_t>(blocks128(a.b_rows)), sf_cols, 2, 64, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tensor_map_2d(&my, a.Y, kBf16Out ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                          kBf16Out ? 2 : 4, static_cast<uint64_t>(a.y_rows), static_cast<uint64_t>(a.N), 32,
                          kBf16Out ? 64 : 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  Params p = {};
  p.M = a.M;
  p.N = a.N;
  p.tiles_m = static_cast<int>((a.M + 255) / 256);
  p.tiles_n = static_cast<int>((a.N + 255) / 256);
  p.nkb = static_cast<int>(blocks128(a.K));
  // kRows: at most one tile per 128-row block of the buffer
  const int64_t m_tiles = kMode == Fp8GemmArgs::kRows ? a.M / 128 : static_cast<int64_t>(p.tiles_m) * a.E;
  const int64_t tiles = m_tiles * p.tiles_n;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  p.num_tiles = static_cast<int>(tiles);
  p.a_oob = static_cast<int>(blocks128(a.a_rows) * 128);
  // 16384 x 6144 bf16 (201 MB): 97 -> 88 us; 67 MB: no change, and its reader may find it there
  p.y_passes = a.y_rows * a.N * (kBf16Out ? 2 : 4) > int64_t{100} << 20 ? 1 : 0;
  p.E = a.E;
  p.counts = a.counts;
  if (a.table) p.t = *a.table;
  p.Y = a.Y;
  p.flags = a.flags;
  p.status = a.status;
  auto kern = fp8_gemm_kernel<kMode, kBf16Out>;
  const void* fn = reinterpret_cast<const void*>(kern);
  const size_t smem = Cfg::kSmemBytes + (kMode == Fp8GemmArgs::kRows ? sizeof(Buffer) : 0);
  cudaError_t e = set_max_dynamic_smem(fn, smem);
  if (e != cudaSuccess) return e;
  // one pair per two SMs that can hold pairs at once
  static std::atomic<int> resident[kFp8CachedDevices];
  int most = fp8_resident_pairs(fn, Cfg::kThreads, smem, resident);
  if (most > kFp8MaxPairs) most = kFp8MaxPairs;
  p.cut0 = 0x7FFFFFFF;
  p.parts = 1;
  if (kMode == Fp8GemmArgs::kDense && !kBf16Out && tiles % most != 0) {
    // the last round's tiles: as many parts as there are pairs for, of at least
    // kMinPart blocks, at most 4 (each waits for the one below)
    const int rem = p.num_tiles % most;
    int parts = most / rem < 4 ? most / rem : 4;
    if (parts > p.nkb / kMinPart) parts = p.nkb / kMinPart;
    if (parts > 1) {
      p.cut0 = p.num_tiles - rem;
      p.parts = parts;
      p.num_tiles += rem * (parts - 1);
    }
  }
  const int pairs = p.num_tiles < most ? p.num_tiles : most;
  return launch_ex(kern, dim3(2 * pairs), dim3(Cfg::kThreads), smem, s, true, ma, mb, msa, msb, my, p);
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t s) {
  if (fp8_stream_applies(a)) return launch_fp8_stream(a, s);
  const bool b = a.yt == AVR_BF16;
  switch (a.mode) {
    case Fp8GemmArgs::kDense: return b ? gemm_t<Fp8GemmArgs::kDense, true>(a, s) : gemm_t<Fp8GemmArgs::kDense, false>(a, s);
    case Fp8GemmArgs::kRows: return b ? gemm_t<Fp8GemmArgs::kRows, true>(a, s) : gemm_t<Fp8GemmArgs::kRows, false>(a, s);
    case Fp8GemmArgs::kTokens:
      return b ? gemm_t<Fp8GemmArgs::kTokens, true>(a, s) : gemm_t<Fp8GemmArgs::kTokens, false>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace avr
