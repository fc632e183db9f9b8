// Tree attention on tcgen05 tensor cores (fp16 / bf16 q; 16-bit or 8-bit
// cache). The work split is in pa_tree.cuh.
//
// A query tile is 128 rows (tree node, query head), so every K/V tile is read
// once for floor(128 / G) nodes. Per 64-key tile and 128-wide head a CTA reads
// 32 KB of a 16-bit cache, which takes its share of HBM about 1400 cycles at
// two CTAs per SM; the two products take 640 tensor-pipe cycles (S = Q K^T
// re-reads Q from shared memory: 8 steps of 48 cycles; O += P V 4 of 64),
// whether the rows are all in use or not. Two CTAs share an SM: one's prologue,
// epilogue and piece switches run under the other's stream. Measured:
//   4 sequences of 131072, trees of 12, group 8: 248 us, HBM (6.7 TB/s);
//   64 of 4096, trees of 16, group 4: 118 us, HBM at 78% of its cycles;
//   48 of 8192, trees of 40, group 8 (two or three query tiles a KV head):
//     303 us; the tensor unit is busy 73% of the cycles (50% in its pipe, the
//     rest on its operands' way), HBM 61%;
//   64 of 4096 over an e4m3 cache, trees of 16, group 8: 143 us, HBM at 34%,
//     70 key tiles a CTA. In long pieces (4 sequences of 131072: 166 tiles a
//     CTA in 247 us, no less than over a 16-bit cache) a tile takes 1.5 us, 2850
//     cycles: the latency of one softmax thread's row of 64 scores, read
//     twice, and of the hand-overs around it. That is some 104 of the 143 us;
//     the rest is start-up and a CTA's 2.7 pieces, each of which waits for Q and
//     for its conversion. Two threads a row (234 us), one pass over the row
//     with registers moved between warpgroups (168) and converters that fetch
//     the codes themselves (164) were slower, as more warps wait on more
//     barriers.
//
//   warps 0, 6  producers: Q tile of each piece and K tiles, V tiles, through
//               the block table into rings of NK and NV stages;
//   warp 1      tensor memory (256 columns: two S tiles of 64, O of head_dim)
//               and, one lane, the MMAs: S(g) before O += P(g-1) V(g-1), so the
//               softmax of a tile runs under the next tile's S;
//   warps 2-5   softmax: thread i owns row i (tensor-memory lane i): its S row,
//               masked by its node's ancestors where the tile reaches into the
//               tree, running max and sum in registers, P (16-bit) over S, O
//               rescaled in tensor memory when the max has moved by more than
//               2^8, and the output or partial at the end of a piece;
//   warps 7-9   (8-bit cache) widen the codes of each stage to fp16 in place
//               and move a bf16 Q tile into fp16, a power of two per row.
// All roles walk the CTA's pieces; stages, S tiles and their barriers are
// counted over all tiles of the CTA, so the rings run on across pieces.
//
// Scores, maxima, sums and O are held in 32 bits. Two things are rounded to 16.
// A softmax weight is, as the second product's operand, while the row's sum takes
// it as it was: it is off by at most half a step, the size of the output's own
// rounding, and in fp16 below 2^-14 by at most 2^-25, which over n such keys can
// add up to n 2^-25 of their values. And over an 8-bit cache a bf16 row of q is,
// into fp16 by a power of two (exact for all that lies within 2^24 of the row's
// largest), since codes are exact in fp16 only. The V scale of a block is taken
// into the weight before that rounding, by a power of two that keeps it below
// 2^15: a row's own, from the blocks that it sees a key of.
//
// A row must not see other branches' values, whatever they hold, but P V
// multiplies every row's weights (0 for those) with every key's values. So
// in tiles that reach into the tree the softmax warps replace values that are
// not finite by 0 in shared memory, note their nodes, and add them to the
// rows that do see them at the end (a sum with a positive weight on an
// infinity or NaN is that infinity or NaN whatever the weight is).
//
// Every mbarrier wait is bounded: on a timeout the kernel records
// PA_ERR_TIMEOUT, lets copies and MMAs in flight finish (bounded), frees
// tensor memory and returns.
#include <math_constants.h>

#include <type_traits>

#include "pa_tcgen05.cuh"
#include "pa_tree.cuh"

namespace pa {

namespace tt {
constexpr int kM = 128;
constexpr int kN = 64;
constexpr int kHalf = kN * 128;       // 64 columns of a K / V tile: 64 rows of 128 bytes
constexpr int kQHalf = kM * 128;
constexpr int kSoftmaxWarp0 = 2;
constexpr int kVWarp = 6;
constexpr int kConvWarp0 = 7;
constexpr int kConvK = 2;              // warps that widen K; one more widens V
constexpr int kConvWarps = kConvK + 1;
constexpr int kQSlots = 3;            // pieces whose Q exponents are kept (8-bit cache)
constexpr int kScaleSlots = 4;        // tiles whose scales are kept (8-bit cache): a K tile's copy is issued after
                                      // the softmax of the tile four before it (NK = 2)
template <int D, bool KV8>
struct Cfg {
  static constexpr int kH = D / 64;            // 64-column halves
  // K / V stage: groups of eight rows of 128 bytes (the swizzle's atom). At
  // head_dim 128 a 16-bit group's two halves lie side by side, so that one copy
  // brings a whole block; codes are widened in place, a row's lower half into
  // the stage's first 8 KB and its upper half over the codes.
  static constexpr int kGroup = D == 128 && !KV8 ? 2048 : 1024;  // distance of groups
  static constexpr int kHalfOff = KV8 ? kHalf : 1024;            // of a group's halves
  // Stages. A V tile waits for the softmax of its keys, a K tile does not.
  static constexpr int NK = D == 64 ? 5 : 2;
  static constexpr int NV = D == 64 ? 6 : 3;
  static constexpr int kStage = kH * kHalf;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kH * kQHalf;
  static constexpr int kOffV = kOffK + NK * kStage;
  static constexpr int kOffBar = kOffV + NV * kStage;
  // barriers
  static constexpr int kBarQFull = 0, kBarQEmpty = 1;
  static constexpr int kBarSoft = 2;  // the four softmax warps
  // P(g) completes barrier g % 2: a wait for tile g then cannot meet tile
  // g - 1's phase, and tile g - 2's is over once S(g) is known to be computed.
  // S(g) computed is its K stage's release, and P(g)'s product its V stage's: the
  // softmax waits on those barriers too (a commit takes the MMA thread 60 to
  // 100 cycles, and it issues without a pause).
  static constexpr int kBarP = 4;
  // 8-bit cache: piece i's Q is in fp16 (i % 3: the MMAs may be two pieces of
  // one tile each ahead of the softmax, which waits for it too).
  static constexpr int kBarQConv = 6;
  static constexpr int kBarKFull = 9, kBarKEmpty = kBarKFull + NK, kBarKCode = kBarKEmpty + NK;
  static constexpr int kBarVFull = kBarKCode + NK, kBarVEmpty = kBarVFull + NV, kBarVCode = kBarVEmpty + NV;
  static constexpr int kNumBars = kBarVCode + NV;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;   // tensor-memory base, the notes' two flags
  // Notes of nodes with values that are not finite, by piece parity (a softmax
  // warp may be one piece ahead of another); before that the scan's scratch.
  static constexpr int kOffPoison = kOffMisc + 16;
  static constexpr int kOffScale = kOffPoison + 2 * kMaxTreeNodes / 8;  // [kScaleSlots][kN / 16] (K, V)
  static constexpr int kOffQExp = kOffScale + (KV8 ? kScaleSlots * (kN / 16) * 8 : 0);
  static constexpr int kSmem = kOffQExp + (KV8 ? kQSlots * kM : 0);
};
static_assert(Cfg<128, true>::kSmem <= 115712 && Cfg<128, false>::kSmem <= 115712, "two CTAs per SM");
constexpr int kTmemCols = 256;
constexpr int kColO = 2 * kN;
template <bool KV8>
__host__ __device__ constexpr int threads() { return KV8 ? 320 : 224; }
static_assert((threads<false>() / 16 + 2) * 8 <= Cfg<64, false>::kSmem - Cfg<64, false>::kOffPoison &&
                  (threads<true>() / 16 + 2) * 8 <= Cfg<128, true>::kSmem - Cfg<128, true>::kOffPoison,
              "the scan's scratch");
}  // namespace tt

// mbar_wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) <= 3.4028235e38f); }

// Zero the 16-bit values of `w` that are not finite; true if there was one.
template <bool BF16>
__device__ __forceinline__ bool strip_not_finite(uint32_t& w) {
  constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  const bool lo = (w & e) == e, hi = ((w >> 16) & e) == e;
  if (lo) w &= 0xffff0000u;
  if (hi) w &= 0x0000ffffu;
  return lo || hi;
}

template <typename T, int BS, int D, bool KV8, bool E5>
__global__ void __launch_bounds__(tt::threads<KV8>(), 2)
    tree_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using namespace tt;
  using C = Cfg<D, KV8>;
  using MT = typename std::conditional<KV8, __half, T>::type;  // the MMA's 16-bit type
  constexpr bool kBf16 = std::is_same<MT, __nv_bfloat16>::value;
  constexpr uint32_t kIdescS = idesc_f16(kM, kN, kBf16, false);
  constexpr uint32_t kIdescO = idesc_f16(kM, D, kBf16, true);
  constexpr int kBlocks = kN / BS;  // blocks of a tile
  constexpr int kThreads = threads<KV8>();
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8 * i; };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_trigger();
  if (threadIdx.x == 0) {
    if ((sbase & 1023u) != 0) record_error(p.status, PA_ERR_ALIGN);
    mbar_init(bar(C::kBarQFull), 1);
    mbar_init(bar(C::kBarQEmpty), 1);
    for (int i = 0; i < kQSlots; ++i) mbar_init(bar(C::kBarQConv + i), kConvWarps);
    mbar_init(bar(C::kBarSoft), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kBarP + i), 4);
    }
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(bar(C::kBarKFull + i), KV8 ? kConvK : 1);
      mbar_init(bar(C::kBarKEmpty + i), 1);
      mbar_init(bar(C::kBarKCode + i), 1);
    }
    for (int i = 0; i < C::NV; ++i) {
      mbar_init(bar(C::kBarVFull + i), 1);
      mbar_init(bar(C::kBarVEmpty + i), 1);
      mbar_init(bar(C::kBarVCode + i), 1);
    }
    p.merge[blockIdx.x].parts = 0;
    fence_barrier_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(&misc[0])), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const TreeRange range = tree_range<kThreads>(p, reinterpret_cast<int64_t*>(smem + C::kOffPoison));
  __syncthreads();  // the scratch becomes the notes
  const uint32_t tmem = misc[0];
  const int G = p.group;
  const int pp = p.tile_rows / G;  // nodes of a query tile

  TreeWalk walk(p, range);
  TreePiece c;
  int g = 0;       // tiles of this CTA so far
  int piece = 0;
  if ((sbase & 1023u) != 0) {
    // (misaligned shared memory, reported above: nothing can run)
  } else if (warp == 0 || warp == kVWarp) {
    // ============================= producers ==============================
    // Issuing a copy takes its warp about 80 cycles, and a wait 200, so K (with
    // Q) and V have a warp each: with one for both, the 8-bit kernel's tiles
    // were spaced by their issue (2000 of 3300 cycles).
    const bool is_v = warp == kVWarp;
    const int ns = is_v ? C::NV : C::NK;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    const int full0 = KV8 ? (is_v ? C::kBarVCode : C::kBarKCode) : (is_v ? C::kBarVFull : C::kBarKFull);
    const int empty0 = is_v ? C::kBarVEmpty : C::kBarKEmpty;
    const uint32_t stage0 = sbase + (is_v ? C::kOffV : C::kOffK) + (KV8 ? kHalf : 0);
    bool bad = false;
    int q_issued = 0;
    while (!bad && walk.next(p, c)) {
      const int32_t* table = p.block_tables + (int64_t)c.seq * p.max_blocks_per_seq;
      const int nblk = (c.kv_len() + BS - 1) / BS;
      // Lane l holds block l of a batch of 32 (8 or 16 tiles); the next batch
      // is requested a batch ahead. Blocks behind the sequence read block 0:
      // their keys are masked and their values zeroed.
      constexpr int kBatch = 32 / kBlocks;
      auto load_batch = [&](int t) -> int {
        const int b = t * kBlocks + lane;
        int id = 0;
        if (b < nblk && t < c.t1) {
          id = table[b];
          if (id < 0 || id >= p.num_blocks) {
            record_error(p.status, PA_ERR_BLOCK_OOB);
            id = -1;
          }
        }
        return id;
      };
      // 8-bit cache: the (K, V) scales of a batch's blocks, 0 where there is
      // none, requested with the batch.
      auto load_scales = [&](int t, int id) -> float2 {
        float2 r = make_float2(0.f, 0.f);
        if (KV8 && !is_v && t * kBlocks + lane < nblk && t < c.t1 && id >= 0)
          r = __ldg(reinterpret_cast<const float2*>(p.kv_scales) + (int64_t)id * p.num_kv_heads + c.kvh);
        return r;
      };
      int id_cur = load_batch(c.t0), id_next = load_batch(c.t0 + kBatch);
      float2 sc_cur = load_scales(c.t0, id_cur), sc_next = make_float2(0.f, 0.f);
      for (int t = c.t0; t < c.t1 && !bad; ++t, ++g) {
        const int in = (t - c.t0) % kBatch;
        if (t > c.t0 && in == 0) {
          id_cur = id_next;
          sc_cur = sc_next;
          id_next = load_batch(t + kBatch);
        }
        if (KV8 && in == kBatch / 2) sc_next = load_scales(t - in + kBatch, id_next);
        const int st = g % ns;
        const uint32_t full = bar(full0 + st);
        if (lane == 0) {
          if (g >= ns && !mbar_wait(bar(empty0 + st), ((g / ns) & 1) ^ 1, p.status)) bad = true;
        }
        bad = __shfl_sync(0xffffffffu, bad, 0);
        if (bad) break;
        if constexpr (KV8) {
          // Group u's scales, for the softmax: published by the arrival below.
          if (!is_v && lane >= in * kBlocks && lane < (in + 1) * kBlocks) {
            float2* to = reinterpret_cast<float2*>(smem + C::kOffScale) + (g % kScaleSlots) * (kN / 16);
#pragma unroll
            for (int i = 0; i < BS / 16; ++i) to[(lane - in * kBlocks) * (BS / 16) + i] = sc_cur;
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(full, KV8 ? kHalf : C::kStage);
        const int id = __shfl_sync(0xffffffffu, id_cur, in * kBlocks + lane % kBlocks);
        if (lane < kBlocks) {
          const int row = (max(id, 0) * p.num_kv_heads + c.kvh) * BS;
          const uint32_t dst = stage0 + st * C::kStage + lane * (BS / 8) * (KV8 ? 1024 : C::kGroup);
          if constexpr (D == 128 && !KV8) tma_load_4d(dst, map, 0, 0, 0, row / 8, full);
          else tma_load_2d(dst, map, 0, row, full);
        }
        if (!is_v && t == c.t0) {
          // Q after the piece's first K tile: its place is free once the
          // previous piece's last S has been computed.
          if (lane == 0) {
            if (piece > 0 && !mbar_wait(bar(C::kBarQEmpty), (piece - 1) & 1, p.status)) {
              bad = true;
            } else {
              mbar_arrive_expect_tx(bar(C::kBarQFull), C::kH * pp * G * 128);
#pragma unroll
              for (int h = 0; h < C::kH; ++h)
                tma_load_3d(sbase + C::kOffQ + h * kQHalf, &qmap, h * 64, c.kvh * G, c.s.q0 + c.qt * pp,
                            bar(C::kBarQFull));
              q_issued = piece + 1;
            }
          }
          bad = __shfl_sync(0xffffffffu, bad, 0);
        }
      }
      ++piece;
    }
    if (bad && lane == 0) {  // copies in flight land before the CTA ends
      if (q_issued > 0) mbar_wait(bar(C::kBarQFull), (q_issued - 1) & 1, nullptr);
      for (int j = max(0, g - ns); j < g; ++j) mbar_wait(bar(full0 + j % ns), (j / ns) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================ MMA =================================
    if (lane == 0) {
      bool bad = false;
      uint32_t last_bar = 0, last_phase = 0;  // the last commit covers every MMA before it
      const uint64_t dq = sdesc_sw128(sbase + C::kOffQ, 16, 1024);
      const uint64_t dk = sdesc_sw128(sbase + C::kOffK, 16, C::kGroup);
      const uint64_t dv = sdesc_sw128(sbase + C::kOffV, C::kHalfOff, C::kGroup);
      auto commit = [&](uint32_t b, int phase) {
        tc_commit(b);
        last_bar = b;
        last_phase = phase & 1;
      };
      auto issue_pv = [&](int j, bool first) -> bool {
        if (!mbar_wait(bar(C::kBarVFull + j % C::NV), (j / C::NV) & 1, p.status)) return false;
        if (!mbar_wait(bar(C::kBarP + (j & 1)), (j >> 1) & 1, p.status)) return false;
        tc_fence_after();
        const uint64_t va = dv + (uint64_t)((j % C::NV) * (C::kStage >> 4));
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)
          tc_mma_f16_ta(tmem + kColO, tmem + (j & 1) * kN + k * 8, va + ((k * 2 * C::kGroup) >> 4), kIdescO,
                        !first || k > 0 ? 1u : 0u);
        commit(bar(C::kBarVEmpty + j % C::NV), j / C::NV);
        return true;
      };
      bool first_prev = false;  // tile g - 1 was its piece's first
      while (!bad && walk.next(p, c)) {
        // The previous piece's last product does not wait for this piece's Q.
        if (g > 0 && !issue_pv(g - 1, first_prev)) bad = true;
        if (!bad && !mbar_wait(KV8 ? bar(C::kBarQConv + piece % kQSlots) : bar(C::kBarQFull),
                                KV8 ? (piece / kQSlots) & 1 : piece & 1, p.status)) bad = true;
        for (int t = c.t0; t < c.t1 && !bad; ++t, ++g) {
          if (!mbar_wait(bar(C::kBarKFull + g % C::NK), (g / C::NK) & 1, p.status)) {
            bad = true;
            break;
          }
          tc_fence_after();
          const uint64_t ka = dk + (uint64_t)((g % C::NK) * (C::kStage >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_f16(tmem + (g & 1) * kN, dq + (((k >> 2) * kQHalf + (k & 3) * 32) >> 4),
                       ka + (((k >> 2) * C::kHalfOff + (k & 3) * 32) >> 4), kIdescS, k > 0);
          commit(bar(C::kBarKEmpty + g % C::NK), g / C::NK);
          if (t + 1 == c.t1) commit(bar(C::kBarQEmpty), piece);
          if (t > c.t0 && !issue_pv(g - 1, first_prev)) bad = true;
          first_prev = t == c.t0;
        }
        ++piece;
      }
      if (!bad && g > 0 && !issue_pv(g - 1, first_prev)) bad = true;
      if (bad && last_bar) mbar_wait(last_bar, last_phase, nullptr);
    }
    __syncwarp();
  } else if (KV8 && warp >= kConvWarp0) {
    // ============================= converters =============================
    if constexpr (KV8) {
      const int ct = threadIdx.x - 32 * kConvWarp0;
      bool bad = false;
      while (!bad && walk.next(p, c)) {
        if (!mbar_wait_warp(bar(C::kBarQFull), piece & 1, p.status)) bad = true;
        if (!bad && std::is_same<T, __nv_bfloat16>::value) {
          // bf16 rows into fp16: x 2^-sh, sh from the row's largest magnitude
          // (then below 2^15), so what lies within 2^24 of it stays exact.
          uint8_t* qexp = smem + C::kOffQExp + piece % kQSlots * kM;
          for (int r = ct; r < kM; r += 32 * kConvWarps) {
            uint8_t* rb = smem + C::kOffQ + r * 128;
            auto chunk = [&](int i) { return reinterpret_cast<uint4*>(rb + (i >> 3) * kQHalf + (((i & 7) ^ (r & 7)) << 4)); };
            float amax = 0.f;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
              const uint4 raw = *chunk(i);
              const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                amax = fmax3(amax, fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u)));
            }
            const uint32_t field = max(16u, __float_as_uint(amax) >> 23);  // exponent field; a tiny row counts as 2^-110
            const float mul = __uint_as_float((268u - min(field, 254u)) << 23);  // 2^(141 - field)
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
              const uint4 raw = *chunk(i);
              uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = MmaOp<__half>::pack(__uint_as_float(w[e] << 16) * mul, __uint_as_float(w[e] & 0xffff0000u) * mul);
              *chunk(i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            qexp[r] = (uint8_t)min(field, 254u);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarQConv + piece % kQSlots));
        // The K warps take 32 rows each, the V warp all 64.
        const bool is_v = ct >= 32 * kConvK;
        const int ns = is_v ? C::NV : C::NK;
        for (int t = c.t0; t < c.t1 && !bad; ++t, ++g) {
          const int st = g % ns;
          if (!mbar_wait_warp(bar((is_v ? C::kBarVCode : C::kBarKCode) + st), (g / ns) & 1, p.status)) {
            bad = true;
            break;
          }
#pragma unroll 1
          for (int r = is_v ? lane : ct; r < kN; r += is_v ? 32 : 32 * kConvK) {
            // A row's codes lie where its widened upper half goes: read whole, then written.
            uint8_t* base = smem + (is_v ? C::kOffV : C::kOffK) + st * C::kStage + r * 128;
            uint4 cr[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) cr[i] = *reinterpret_cast<const uint4*>(base + kHalf + ((i ^ (r & 7)) << 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t o[8];
              fp8x4_to_f16x4<E5>(cr[i].x, o[0], o[1]);
              fp8x4_to_f16x4<E5>(cr[i].y, o[2], o[3]);
              fp8x4_to_f16x4<E5>(cr[i].z, o[4], o[5]);
              fp8x4_to_f16x4<E5>(cr[i].w, o[6], o[7]);
              uint8_t* rb = base + (i >> 2) * kHalf;
              const int cc = 2 * (i & 3);
              *reinterpret_cast<uint4*>(rb + ((cc ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(rb + (((cc + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar((is_v ? C::kBarVFull : C::kBarKFull) + st));
        }
        ++piece;
      }
    }
  } else {
    // ============================== softmax ===============================
    const int q = warp & 3;
    const int row = q * 32 + lane;  // row of the tile = tensor-memory lane
    const int tid = threadIdx.x - 32 * kSoftmaxWarp0;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    bool bad = false;
    for (int i = tid; i < 2 * kMaxTreeNodes / 32; i += 128) reinterpret_cast<uint32_t*>(smem + C::kOffPoison)[i] = 0;
    if (tid < 2) misc[1 + tid] = 0;
    int syncs = 0;
    auto soft_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kBarSoft));
      return mbar_wait_warp(bar(C::kBarSoft), syncs++ & 1, p.status);
    };
    bad = !soft_sync();
    while (!bad && walk.next(p, c)) {
      const int32_t* parents = p.parents + c.s.q0;
      const int32_t* table = p.block_tables + (int64_t)c.seq * p.max_blocks_per_seq;
      const int kv_len = c.kv_len(), ctx = c.s.ctx;
      const int node = c.qt * pp + row / G;
      const bool used = row < pp * G && node < c.s.nodes;
      const bool live = q * 32 < pp * G && c.qt * pp + q * 32 / G < c.s.nodes;  // the warp has a row in use
      const bool tree = c.t1 * kN > ctx;  // the piece reaches into the tree
      uint32_t* poison = reinterpret_cast<uint32_t*>(smem + C::kOffPoison) + (piece & 1) * (kMaxTreeNodes / 32);
      volatile uint32_t* poisoned = &misc[1 + (piece & 1)];
      if (tree) tree_check_parents<128>(p, c, tid);
      float m = -CUDART_INF_F, l = 0.f;
      // 8-bit cache: scores are scaled to log2 units before the max.
      const float sl2 = KV8 ? 1.f : p.scale_log2;
      float rf = p.scale_log2;
      constexpr int kKapUnset = 1 << 20;
      int kap = kKapUnset;
      float pw = 1.f;
      if constexpr (KV8 && std::is_same<T, __nv_bfloat16>::value) {
        if (!mbar_wait_warp(bar(C::kBarQConv + piece % kQSlots), (piece / kQSlots) & 1, p.status)) bad = true;
        rf = ldexpf(p.scale_log2, (int)smem[C::kOffQExp + piece % kQSlots * kM + row] - 141);
      }
      for (int t = c.t0; t < c.t1 && !bad; ++t, ++g) {
        const int k0 = t * kN;
        const uint32_t ts = tl + (g & 1) * kN, to = tl + kColO;
        if (!mbar_wait_warp(bar(C::kBarKEmpty + g % C::NK), (g / C::NK) & 1, p.status)) {
          bad = true;
          break;
        }
        tc_fence_after();
        if (live) {
          // Keys that the row sees, in tiles that reach into the tree.
          uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
          const bool masked = k0 + kN > ctx;
          if (masked) {
            const int first = k0 - ctx;  // node of the tile's first key (below 0: context)
            seen[0] = tree_ancestors(parents, used ? node : -1, first);
            seen[1] = tree_ancestors(parents, used ? node : -1, first + 32);
            if (first < 0) {
              seen[0] |= first > -32 ? (1u << -first) - 1u : 0xffffffffu;
              if (first < -32) seen[1] |= (1u << (-first - 32)) - 1u;
            }
            __syncwarp();  // (the walks differ in length)
          }
          auto mask = [&](uint32_t (&v)[32], uint32_t bits) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((bits >> i) & 1u)) v[i] = __float_as_uint(-CUDART_INF_F);
          };
          // alpha takes the row to a larger maximum: only when it has moved by
          // more than 2^8 (weights stay below 256), or from nothing.
          float alpha = 1.f;
          auto update_max = [&](float mx) {
            if (m == -CUDART_INF_F) {
              m = mx;
            } else if ((mx - m) * sl2 > 8.f) {
              alpha = fast_exp2((m - mx) * sl2);
              m = mx;
            }
          };
          // O times f, once the previous product has been added to it.
          auto rescale = [&](float f) -> bool {
            if (t == c.t0 || !__any_sync(0xffffffffu, f != 1.f)) return true;
            if (!mbar_wait_warp(bar(C::kBarVEmpty + (g - 1) % C::NV), ((g - 1) / C::NV) & 1, p.status)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              uint32_t o[16];
              tmem_ld16(to + i * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(to + i * 16, o);
            }
            return true;
          };
          uint64_t rs2 = f2_pack(0.f, 0.f);
          if constexpr (!KV8) {
            uint32_t sr[2][32];
            tmem_ld32(ts, sr[0]);
            tmem_ld32(ts + 32, sr[1]);
            tmem_ld_wait();
            if (masked) mask(sr[0], seen[0]), mask(sr[1], seen[1]);
            float mx = -CUDART_INF_F;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                mx = fmax3(mx, __uint_as_float(sr[h][i]), __uint_as_float(sr[h][i + 1]));
            update_max(mx);
            if (!rescale(alpha)) {
              bad = true;
              break;
            }
            const float neg = m == -CUDART_INF_F ? 0.f : -m * sl2;
            const uint64_t sl2x2 = f2_pack(sl2, sl2), negx2 = f2_pack(neg, neg);
            uint32_t pk[32];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[h][i]), __uint_as_float(sr[h][i + 1])), sl2x2, negx2), x0,
                          x1);
                const float a = fast_exp2(x0), b = fast_exp2(x1);
                rs2 = f2_add(rs2, f2_pack(a, b));
                pk[h * 16 + i / 2] = MmaOp<MT>::pack(a, b);
              }
            tmem_st32(ts, pk);
          } else {
            // Two passes over the S row, 32 keys at a time (registers): the
            // scores of 16-key group u are s * f_u, f_u >= 0, so a group's
            // largest is its raw largest times f_u exactly.
            const float2* scales = reinterpret_cast<const float2*>(smem + C::kOffScale) + (g % kScaleSlots) * (kN / 16);
            // Groups that the row sees no key of stay out, here and below: another
            // branch's block may have any V scale. (A seen group's scale is
            // that of values the row sees.)
            float vmax = 0.f;
#pragma unroll
            for (int u = 0; u < kN / 16; ++u)
              if ((seen[u >> 1] >> (16 * (u & 1))) & 0xffffu) vmax = fmaxf(vmax, scales[u].y);
            float kap_r = 1.f;  // 2^(new kap - old kap) where kap drops
            if (vmax > 0.f) {
              // 2^kap brings the largest V scale seen so far below 2^7.
              const int ex = (int)((__float_as_uint(vmax) >> 23) & 0xffu) - 126;
              const int kmax = min(7 - ex, 127);
              if (kmax < kap) {
                if (kap != kKapUnset) kap_r = __uint_as_float((uint32_t)(max(kmax - kap, -126) + 127) << 23);
                kap = kmax;
                pw = __uint_as_float((uint32_t)(kmax + 127) << 23);
              }
            }
            float mx = -CUDART_INF_F;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32];
              tmem_ld32(ts + h * 32, v);
              const float f0 = scales[h * 2].x * rf, f1 = scales[h * 2 + 1].x * rf;
              tmem_ld_wait();
              if (masked) mask(v, h ? seen[1] : seen[0]);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                float x = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                  x = fmax3(x, __uint_as_float(v[u * 16 + i]), __uint_as_float(v[u * 16 + i + 1]));
                mx = fmaxf(mx, x == -CUDART_INF_F ? x : x * (u ? f1 : f0));  // (-inf times a scale of 0)
              }
            }
            update_max(mx);
            if (!rescale(alpha * kap_r)) {  // O takes the drop of kap too, l does not
              bad = true;
              break;
            }
            const float neg = m == -CUDART_INF_F ? 0.f : -m;
            const uint64_t negx2 = f2_pack(neg, neg);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32], pk[16];
              tmem_ld32(ts + h * 32, v);
              const float2 s0 = scales[h * 2], s1 = scales[h * 2 + 1];
              const uint32_t bits = h ? seen[1] : seen[0];
              const float f0 = s0.x * rf, f1 = s1.x * rf;
              const float w0 = bits & 0xffffu ? s0.y * pw : 0.f, w1 = bits >> 16 ? s1.y * pw : 0.f;
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float f = i < 16 ? f0 : f1, w = i < 16 ? w0 : w1;
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), f2_pack(f, f), negx2), x0,
                          x1);
                float a = fast_exp2(x0), b = fast_exp2(x1);
                if (masked) {  // (a masked score may be anything)
                  a = (bits >> i) & 1u ? a : 0.f;
                  b = (bits >> (i + 1)) & 1u ? b : 0.f;
                }
                rs2 = f2_add(rs2, f2_pack(a, b));
                pk[i / 2] = MmaOp<MT>::pack(a * w, b * w);
              }
              tmem_st16(ts + h * 16, pk);  // (columns already read)
            }
          }
          float rs0, rs1;
          f2_unpack(rs2, rs0, rs1);
          l = l * alpha + (rs0 + rs1);
          tmem_st_wait();
        }
        // Values behind the sequence become 0, and those in the tree that are
        // not finite are taken out.
        if (k0 + kN > ctx) {
          const int sv = g % C::NV;
          if (!mbar_wait_warp(bar(C::kBarVFull + sv), (g / C::NV) & 1, p.status)) {
            bad = true;
            break;
          }
          const int first = max(ctx - k0, 0);
          uint8_t* vst = smem + C::kOffV + sv * C::kStage;
          for (int i = tid; i < (kN - first) * 8 * C::kH; i += 128) {
            const int r = first + i / (8 * C::kH), x = i % (8 * C::kH);
            uint4* at = reinterpret_cast<uint4*>(vst + (r >> 3) * C::kGroup + (x >> 3) * C::kHalfOff + (r & 7) * 128 + (x & 7) * 16);
            if (k0 + r >= kv_len) {
              *at = make_uint4(0, 0, 0, 0);
            } else {
              uint4 w = *at;
              const bool b0 = strip_not_finite<kBf16>(w.x), b1 = strip_not_finite<kBf16>(w.y);
              const bool b2 = strip_not_finite<kBf16>(w.z), b3 = strip_not_finite<kBf16>(w.w);
              if (b0 || b1 || b2 || b3) {
                *at = w;
                const int nd = k0 + r - ctx;
                atomicOr(&poison[nd >> 5], 1u << (nd & 31));
                *poisoned = 1;
              }
            }
          }
          fence_async_shared();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarP + (g & 1)));
      }
      if (bad || !mbar_wait_warp(bar(C::kBarVEmpty + (g - 1) % C::NV), ((g - 1) / C::NV) & 1, p.status)) break;
      tc_fence_after();
      // Every warp's notes are made once all have handed over their last P
      // (the next phase of that barrier needs this warp's next tile but one).
      if (tree && !mbar_wait_warp(bar(C::kBarP + ((g - 1) & 1)), ((g - 1) >> 1) & 1, p.status)) break;
      if (tree && *poisoned) {
        // The values taken out above, added for the rows that see their node.
        if (live) {
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t o[16];
            tmem_ld16(tl + kColO + cc * 16, o);
            tmem_ld_wait();
            for (int a = used ? node : -1; a >= 0;) {
              const int pos = ctx + a, id = (poison[a >> 5] >> (a & 31)) & 1u ? table[pos / BS] : -1;
              if (id >= 0 && id < p.num_blocks) {
                const int64_t at = (((int64_t)id * p.num_kv_heads + c.kvh) * BS + pos % BS) * D + cc * 16;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float v;
                  if constexpr (KV8) {
                    uint32_t x0, x1;
                    fp8x4_to_f16x4<E5>(static_cast<const uint8_t*>(p.v_cache)[at + i], x0, x1);
                    v = __half2float(__ushort_as_half((unsigned short)(x0 & 0xffffu)));
                  } else {
                    v = to_f32(static_cast<const T*>(p.v_cache)[at + i]);
                  }
                  if (not_finite(v)) o[i] = __float_as_uint(__uint_as_float(o[i]) + v);
                }
              }
              const int up = __ldg(parents + a);
              a = up < a ? up : -1;
            }
            __syncwarp();
            tmem_st16(tl + kColO + cc * 16, o);
          }
          tmem_st_wait();
        }
        if (!soft_sync()) break;  // read by all
        if (tid < kMaxTreeNodes / 32) poison[tid] = 0;
        if (tid == 0) *poisoned = 0;
        if (!soft_sync()) break;
      }
      const bool whole = c.whole();
      if (c.t0 == 0 && !whole && tid == 0) tree_note_merge(p, range, c);
      if (live) {
        // (1 / l and 1 / pw apart: l * pw overflows for V scales near 2^-120)
        const float f = whole ? 1.f / l : 1.f, ipw = 1.f / pw;
        auto val = [&](uint32_t x) { return KV8 ? __uint_as_float(x) * f * ipw : __uint_as_float(x) * f; };
        const int head = c.kvh * G + row - (row / G) * G;
        T* out = static_cast<T*>(p.out) + ((int64_t)(c.s.q0 + node) * p.num_q_heads + head) * D;
        const int64_t slot = (int64_t)tree_slot(c) * kM + row;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(tl + kColO + cc * 32, o);
          tmem_ld_wait();
          if (used && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 w;
              uint32_t* x = &w.x;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[j] = MmaOp<T>::pack(val(o[i + 2 * j]), val(o[i + 2 * j + 1]));
              *reinterpret_cast<uint4*>(out + cc * 32 + i) = w;
            }
          } else if (used) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(reinterpret_cast<float4*>(p.part_o + slot * D + cc * 32 + i),
                     make_float4(val(o[i]), val(o[i + 1]), val(o[i + 2]), val(o[i + 3])));
          }
        }
        if (used && !whole) __stcg(reinterpret_cast<float2*>(p.part_ml + slot * 2), make_float2(m * sl2, l));
        __syncwarp();
        tc_fence_before();
      }
      ++piece;
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <typename T, int BS, int D, bool KV8, bool E5>
static int run_tree_tc(const TreeParams& p, int ctas, pa_dtype dt, cudaStream_t stream) {
  CUtensorMap qmap, kmap, vmap;
  const int G = p.group;
  // q as [total_q][heads][head_dim]: one box is 64 columns of G heads of the tile's nodes.
  int rc = make_3d_tensor_map(&qmap, p.q, p.total_q, p.num_q_heads, D, dt, p.tile_rows / G, G, 64);
  if (rc != PA_OK) return rc;
  const int64_t rows = (int64_t)p.num_blocks * p.num_kv_heads * BS;
  for (int i = 0; i < 2; ++i) {
    const void* pool = i ? p.v_cache : p.k_cache;
    CUtensorMap* map = i ? &vmap : &kmap;
    rc = KV8 ? make_u8_tensor_map(map, pool, rows, D, BS)
             : D == 128 ? make_kv_group_map(map, pool, rows, BS) : make_kv_tensor_map(map, pool, rows, D, dt, BS);
    if (rc != PA_OK) return rc;
  }
  auto kern = tree_tc_kernel<T, BS, D, KV8, E5>;
  constexpr int smem = tt::Cfg<D, KV8>::kSmem;
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem) != PA_OK) return PA_ERR_CUDA;
  kern<<<ctas, tt::threads<KV8>(), smem, stream>>>(qmap, kmap, vmap, p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename T, int BS>
static int run_tree_tc_bs(const TreeParams& p, int ctas, pa_dtype dt, cudaStream_t stream) {
  if (p.kv_scales)
    return p.kv_fmt == PA_KV_E5M2 ? run_tree_tc<T, BS, 128, true, true>(p, ctas, dt, stream)
                                  : run_tree_tc<T, BS, 128, true, false>(p, ctas, dt, stream);
  return p.head_dim == 64 ? run_tree_tc<T, BS, 64, false, false>(p, ctas, dt, stream)
                          : run_tree_tc<T, BS, 128, false, false>(p, ctas, dt, stream);
}

int launch_tree_tc(const TreeParams& p, int ctas, pa_dtype dt, cudaStream_t stream) {
  if (dt == PA_BF16)
    return p.block_size == 16 ? run_tree_tc_bs<__nv_bfloat16, 16>(p, ctas, dt, stream)
                              : run_tree_tc_bs<__nv_bfloat16, 32>(p, ctas, dt, stream);
  return p.block_size == 16 ? run_tree_tc_bs<__half, 16>(p, ctas, dt, stream)
                            : run_tree_tc_bs<__half, 32>(p, ctas, dt, stream);
}

}  // namespace pa
