// Verification of drafted tokens against the target's probabilities.
//
// At a kept node with target row p and draft row q, its children are tried in
// node order. With w_0 = p and S_0 = 1, child t (token x) is kept when
//   u q(x) S_{t-1} < w_{t-1}(x),
// and refused otherwise, which leaves
//   w_t = max(0, w_{t-1} - S_{t-1} q),  S_t = sum w_t.
// Since max(max(a, 0) - b, 0) = max(a - b, 0) for b >= 0, this is
//   w_t = max(0, p - C_t q),  C_t = S_0 + .. + S_{t-1}:
// any number of refusals is one pass over the two rows, never a stored
// residual. Without q (drafts are certain: q is 1 at the child's token) a
// refusal sets w(x) to 0 and S drops by it. Where no child is kept, the next
// token is the smallest y with w(0) + .. + w(y) > u' sum w.
//
// The token is a whole number that has to come out the same whatever the
// order of the sum, so sums are taken over integers: p - C q is rounded to a
// multiple of 2^-43 (2^18 weights fit 61 bits), and integer sums do not depend
// on their order. Double arithmetic runs at a fraction of the rate, so the
// difference is taken as a float and its rounding error, and split into two
// whole numbers by adding and taking away 1.5 * 2^23, two entries an
// instruction.
//
// A sequence is one cluster of 1 to 8 CTAs, each with a slice of the
// vocabulary; all of them walk the tree by themselves and exchange only sums.
// A warp sums two chunks of 512 entries at a time (16 bytes a load, the chunks'
// loads all in flight) and every chunk's sum is kept, so the entry where the
// running sum passes the threshold takes a second look at one chunk only. 96
// trees over 131072 fp32 tokens take 48 us (100 MB of rows are 15 us of HBM):
// a sequence makes one to four passes one after another, some 9 us each, and
// its start, its exchanges and the draw take 8 us more. A pass is bound by the
// latency of its loads: what is in flight waits in registers, which at two CTAs
// an SM is too little to fill HBM (busy 22%) or to issue without a pause (34%
// of the cycles). One chunk at a time took 61 us, a split of p and C q each 54,
// doubles and one CTA a sequence 1018. With few sequences it is the latency of
// the dependent loads and cluster barriers (4 chains over 32000 tokens: 9 us).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace cg = cooperative_groups;

constexpr int kVerifyMaxNodes = 1024;
constexpr int kVerifyMaxVocab = 1 << 18;
constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyChunk = 512;
constexpr int kVerifyMaxChunks = kVerifyMaxVocab / kVerifyChunk + 1;  // + 1: a row may start inside a 16-byte line
constexpr int kVerifyMaxCluster = 8;
constexpr int kVerifyLow = 21;                           // bits of a weight's lower part
constexpr double kVerifyUnit = 1.0 / 8796093022208.0;  // 2^-43
constexpr unsigned kAll = 0xffffffffu;

struct VerifyParams {
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* cu_q_lens;
  const int32_t* parents;
  const float* u_accept;
  const float* u_sample;
  int64_t target_stride, draft_stride;
  int32_t total_q, max_q_len, vocab, max_path_len;
  int32_t* path;
  int32_t* path_lens;
  int32_t* next_tokens;
  int* status;
};

// NaN counts as 0; values are held to [0, 1].
template <typename T>
__device__ __forceinline__ float prob(T x) { return __saturatef(to_f32(x)); }

// What C is: nothing refused yet (w = p), one refusal (C = 1), or more.
enum VerifyMode { kVerifyPlain, kVerifyOne, kVerifyMore };

// Two values x in [-1, 1] as hi * 2^21 + lo in units of 2^-43, |lo| <= 2^20;
// both above kMagicBits, and lo on top of base's bits (kMagic and whole numbers).
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
constexpr int kMagicBits = 0x4b400000;
__device__ __forceinline__ uint64_t both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ void split2(uint64_t x, uint64_t base, uint64_t& hi, uint64_t& lo) {
  hi = f2_fma(x, both(4194304.f), both(kMagic));
  const uint64_t rest = f2_fma(x, both(4194304.f), f2_fma(hi, both(-1.f), both(kMagic)));  // exact, at most 1/2
  lo = f2_fma(rest, both(2097152.f), base);
}

// max(0, p - C q) of two entries in units of 2^-43 as hi * 2^21 + lo, hi >= 0,
// |lo| < 2^21, added to h and l. C = c + cl (cl: what a float of C leaves
// over). Differences are taken in floats and their rounding errors, exact
// floats too (p - d - m), go into the lower part.
template <int MODE>
__device__ __forceinline__ void add_weights(float p0, float p1, float q0, float q1, float c, float cl, int& h, int& l) {
  const uint64_t p = f2_pack(p0, p1), q = f2_pack(q0, q1);
  const uint64_t minus = both(-1.f);
  uint64_t d = p, base = both(kMagic), hi, lo;
  if constexpr (MODE == kVerifyOne) {
    d = f2_fma(q, minus, p);
    base = f2_fma(f2_fma(q, minus, f2_fma(d, minus, p)), both(8796093022208.f), base);
  } else if constexpr (MODE == kVerifyMore) {
    const uint64_t m = f2_fma(both(c), q, both(0.f));  // C q = m + me
    const uint64_t me = f2_fma(both(cl), q, f2_fma(both(c), q, f2_fma(m, minus, both(0.f))));
    d = f2_fma(m, minus, p);
    const uint64_t e = f2_fma(m, minus, f2_fma(d, minus, p));
    base = f2_fma(f2_fma(me, minus, e), both(8796093022208.f), base);
    float d0, d1;
    f2_unpack(d, d0, d1);
    d = f2_pack(fmaxf(d0, -1.f), fmaxf(d1, -1.f));
  }
  split2(d, base, hi, lo);
  float t0, t1, s0, s1;
  f2_unpack(hi, t0, t1);
  f2_unpack(lo, s0, s1);
  auto add = [&](float pv, float qv, float t, float s) {
    const int a = __float_as_int(t) - kMagicBits, b = __float_as_int(s) - kMagicBits;
    // m may pass p by a rounding although C q < p: the parts decide.
    const bool some = MODE == kVerifyPlain || (MODE == kVerifyOne ? pv > qv : a > 0 || (a == 0 && b > 0));
    h += some ? a : 0;
    l += some ? b : 0;
  };
  add(p0, q0, t0, s0);
  add(p1, q1, t1, s1);
}

template <int MODE>
__device__ __forceinline__ void add_weight(float p, float q, float c, float cl, int& h, int& l) {
  add_weights<MODE>(p, 0.f, q, 0.f, c, cl, h, l);
}

__device__ __forceinline__ long long joined(int hi, int lo) { return ((long long)hi << kVerifyLow) + lo; }

template <typename T>
__device__ __forceinline__ float entry(const uint4& raw, int i) {
  return prob(reinterpret_cast<const T*>(&raw)[i]);
}

// The sums of a slice's chunks, one warp a chunk at a time; returns this
// warp's share of their total.
template <typename T, int MODE>
__device__ __forceinline__ long long slice_sums(const T* a, const T* b, int lead, int V, float c, float cl, int c_lo,
                                                int c_hi, long long* chunk_sum) {
  constexpr int N = 16 / sizeof(T), kLoads = kVerifyChunk / (32 * N);
  const int lane = threadIdx.x & 31;
  const bool line =
      MODE == kVerifyPlain || ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
  long long mine = 0;
  auto done = [&](int k, int h, int l) {
    // 512 entries: h at most 2^31 (as an unsigned sum), l below 2^30 either way.
    const long long s = ((long long)__reduce_add_sync(kAll, (unsigned)h) << kVerifyLow) + __reduce_add_sync(kAll, l);
    if (lane == 0) chunk_sum[k - c_lo] = s;
    mine += s;
  };
  auto whole = [&](int k) { return k < c_hi && k * kVerifyChunk >= lead && (k + 1) * kVerifyChunk - lead <= V; };
  // W whole chunks, their loads all in flight.
  auto chunks = [&](int k, auto W) {
    uint4 x[W.value][kLoads], z[W.value][kLoads];
#pragma unroll
    for (int w = 0; w < W.value; ++w)
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int y = (k + w * kVerifyWarps) * kVerifyChunk - lead + (u * 32 + lane) * N;
        x[w][u] = __ldg(reinterpret_cast<const uint4*>(a + y));
        if constexpr (MODE != kVerifyPlain) z[w][u] = __ldg(reinterpret_cast<const uint4*>(b + y));
      }
#pragma unroll
    for (int w = 0; w < W.value; ++w) {
      int h = 0, l = 0;
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
#pragma unroll
        for (int i = 0; i < N; i += 2)
          add_weights<MODE>(entry<T>(x[w][u], i), entry<T>(x[w][u], i + 1),
                            MODE == kVerifyPlain ? 0.f : entry<T>(z[w][u], i),
                            MODE == kVerifyPlain ? 0.f : entry<T>(z[w][u], i + 1), c, cl, h, l);
      done(k + w * kVerifyWarps, h, l);
    }
  };
#pragma unroll 1
  for (int k = c_lo + (threadIdx.x >> 5); k < c_hi; k += 2 * kVerifyWarps) {
    int odd = k;  // first chunk of the two that is not whole
    if (line && whole(k)) {
      odd = k + kVerifyWarps;
      if (whole(odd)) {
        chunks(k, std::integral_constant<int, 2>());
        continue;
      }
      chunks(k, std::integral_constant<int, 1>());
    }
    // The row's ends, and rows whose 16-byte lines do not match.
#pragma unroll 1
    for (; odd < c_hi && odd <= k + kVerifyWarps; odd += kVerifyWarps) {
      int h = 0, l = 0;
#pragma unroll 4
      for (int e = lane; e < kVerifyChunk; e += 64) {
        float v[2], u[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int y = odd * kVerifyChunk - lead + e + 32 * i;
          const bool in = y >= 0 && y < V;
          v[i] = in ? prob(a[y]) : 0.f;
          if (MODE != kVerifyPlain && in) u[i] = prob(b[y]);
        }
        add_weights<MODE>(v[0], v[1], u[0], u[1], c, cl, h, l);
      }
      done(odd, h, l);
    }
  }
  return mine;
}

// CTAs an SM: two where two rows or 32-bit ones are summed (16-bit rows with draft
// rows: a third has to spill and takes 51.8 us where two take 47.8 for 96 trees
// over 131072, and as long for 64 over 100003 and 32000), four for one 16-bit row.
template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads, sizeof(T) == 4 || DRAFT ? 2 : 4) verify_kernel(const VerifyParams p) {
  constexpr int kMine = kVerifyChunk / 32;
  __shared__ int16_t parent[kVerifyMaxNodes];
  __shared__ int tok[kVerifyMaxNodes];
  __shared__ float px[kVerifyMaxNodes], qx[kVerifyMaxNodes], ua[kVerifyMaxNodes];
  __shared__ bool again[kVerifyMaxNodes];  // an earlier sibling has the same token
  __shared__ long long chunk_sum[kVerifyMaxChunks];
  __shared__ long long slice_sum[2][kVerifyMaxCluster];  // every CTA's, written by it
  __shared__ unsigned long long acc;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int seq = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto started = cluster.barrier_arrive();  // peers' shared memory may be written once all have arrived
  int32_t* path = p.path + (int64_t)seq * p.max_path_len;
  const int q0 = p.cu_q_lens[seq];
  const int64_t n64 = (int64_t)p.cu_q_lens[seq + 1] - q0;
  const bool bad_len = n64 < 0 || q0 < 0 || q0 + n64 > p.total_q || n64 > p.max_q_len;
  const int n = bad_len ? 0 : (int)n64;
  bool bad_tree = false;
  for (int j = tid; j < n; j += kVerifyThreads) {
    const int up = p.parents[q0 + j], t = p.tokens[q0 + j];
    ua[j] = p.u_accept[q0 + j];
    bad_tree |= up < -1 || up >= j || (j == 0 && up != -1);
    const bool real = t >= 0 && t < p.vocab && up >= 0 && up < j;
    parent[j] = real ? (int16_t)up : (int16_t)-1;  // a node without a token is nobody's child
    tok[j] = t;
    px[j] = real ? prob(static_cast<const T*>(p.target)[(int64_t)(q0 + up) * p.target_stride + t]) : 0.f;
    if constexpr (DRAFT)
      qx[j] = real ? prob(static_cast<const T*>(p.draft)[(int64_t)(q0 + up) * p.draft_stride + t]) : 0.f;
  }
  bad_tree = __syncthreads_or(bad_tree);
  cluster.barrier_wait(std::move(started));
  if (bad_len || bad_tree || n == 0) {  // (the same in every CTA of the cluster)
    if (rank == 0) {
      if (tid == 0 && (bad_len || bad_tree)) record_error(p.status, bad_len ? PA_ERR_SEQLEN : PA_ERR_ARG);
      for (int k = tid; k < p.max_path_len; k += kVerifyThreads) path[k] = -1;
      if (tid == 0) p.path_lens[seq] = 0, p.next_tokens[seq] = -1;
    }
    return;
  }
  if constexpr (!DRAFT) {
    for (int j = tid; j < n; j += kVerifyThreads) {
      bool same = false;
      const int up = parent[j], t = tok[j];
      if (up >= 0)
        for (int i = up + 1; i < j; ++i) same |= parent[i] == up && tok[i] == t;
      again[j] = same;
    }
    __syncthreads();
  }

  auto row_a = [&](int r) { return static_cast<const T*>(p.target) + (int64_t)(q0 + r) * p.target_stride; };
  auto row_b = [&](int r) -> const T* {
    if constexpr (DRAFT) return static_cast<const T*>(p.draft) + (int64_t)(q0 + r) * p.draft_stride;
    return nullptr;
  };
  // Chunks are counted from the 16-byte line in which the target's row starts.
  auto lead_of = [&](const T* a) { return (int)((reinterpret_cast<uintptr_t>(a) & 15) / sizeof(T)); };
  int sums = 0, c_lo = 0;
  // The sum of w at row r over the vocabulary; this CTA's chunks' sums stay in
  // chunk_sum. take_out (without a draft row): r's children were refused.
  auto total = [&](int r, double C, bool take_out) -> long long {
    const T* a = row_a(r);
    const T* b = row_b(r);
    const float cm = (float)C, cl = (float)(C - (double)cm);
    const int lead = lead_of(a), chunks = (p.vocab + lead + kVerifyChunk - 1) / kVerifyChunk;
    c_lo = chunks * rank / ranks;
    const int c_hi = chunks * (rank + 1) / ranks;
    if (tid == 0) acc = 0;
    __syncthreads();
    const long long mine =
        C == 0.0 ? slice_sums<T, kVerifyPlain>(a, a, lead, p.vocab, cm, cl, c_lo, c_hi, chunk_sum)
        : C == 1.0 ? slice_sums<T, DRAFT ? kVerifyOne : kVerifyPlain>(a, b, lead, p.vocab, cm, cl, c_lo, c_hi, chunk_sum)
                   : slice_sums<T, DRAFT ? kVerifyMore : kVerifyPlain>(a, b, lead, p.vocab, cm, cl, c_lo, c_hi, chunk_sum);
    if (lane == 0) atomicAdd(&acc, (unsigned long long)mine);
    __syncthreads();
    if (!DRAFT && take_out) {
      for (int j = r + 1 + tid; j < n; j += kVerifyThreads) {
        if (parent[j] != r || again[j]) continue;
        const int c = (tok[j] + lead) / kVerifyChunk;
        if (c < c_lo || c >= c_hi) continue;
        int hi = 0, lo = 0;
        add_weight<kVerifyPlain>(px[j], 0.f, 0.f, 0.f, hi, lo);
        const unsigned long long w = (unsigned long long)-joined(hi, lo);
        atomicAdd(reinterpret_cast<unsigned long long*>(&chunk_sum[c - c_lo]), w);
        atomicAdd(&acc, w);
      }
      __syncthreads();
    }
    long long* here = slice_sum[sums & 1];  // (two in turn: a slow CTA may still be reading the last ones)
    ++sums;
    if (tid < ranks) *cluster.map_shared_rank(&here[rank], tid) = (long long)acc;
    cluster.sync();
    long long all = 0;
    for (int i = 0; i < ranks; ++i) all += here[i];
    return all;
  };

  // ---- the walk: every warp of every CTA takes the same steps ----
  int at = 0, len = 1;
  double C;
  if (rank == 0 && tid == 0) path[0] = 0;
  while (true) {
    double S = 1.0;
    C = 0.0;
    int step = -1;
    bool stale = false;  // S has to be summed before it is used
    for (int base = at + 1; base < n && step < 0 && len < p.max_path_len; base += 32) {
      unsigned kids = __ballot_sync(kAll, base + lane < n && parent[base + lane] == at);
      while (kids) {
        const int j = base + __ffs(kids) - 1;
        kids &= kids - 1;
        if constexpr (DRAFT) {
          if (C == 0.0) {
            // u q < p: one rounding keeps the sign, 2^64 times as large also that of
            // subnormal numbers.
            constexpr float kUp = 18446744073709551616.f;
            if (fmaf(ua[j], qx[j] * kUp, -px[j] * kUp) < 0.f) {
              step = j;
              break;
            }
          } else {
            // S is put off until it decides: from the second sum on it is at most
            // the last one, so a child that would be kept with that is kept.
            // (Not so the first, C = 1: a row may sum to more than 1.)
            const double w = fmax(0.0, (double)px[j] - C * (double)qx[j]);
            if (stale && (C == 1.0 || !((double)ua[j] * (double)qx[j] * S < w)))
              S = (double)total(at, C, false) * kVerifyUnit;
            if ((double)ua[j] * (double)qx[j] * S < w) {
              step = j;
              break;
            }
          }
          C += S;
          stale = true;
        } else {
          const double w = again[j] ? 0.0 : (double)px[j];
          if ((double)ua[j] * S < w) {
            step = j;
            break;
          }
          S -= w;
        }
      }
    }
    if (step < 0) break;
    at = step;
    if (rank == 0 && tid == 0) path[len] = at;
    ++len;
  }

  // ---- the next token ----
  bool take_out = !DRAFT && len < p.max_path_len;  // a full path's last node did not try its children
  long long all = total(at, C, take_out);
  if (all <= 0) {  // nothing left after the refusals: drawn from the target itself
    C = 0.0;
    take_out = false;
    all = total(at, C, false);
  }
  const float us = fminf(__saturatef(p.u_sample[seq]), 0.99999994f);
  const long long tau = (long long)((double)us * (double)all);
  const long long* slice = slice_sum[(sums - 1) & 1];
  long long run = 0;
  for (int i = 0; i < rank; ++i) run += slice[i];
  if (warp == 0 && run <= tau && tau < run + slice[rank]) {
    const T* a = row_a(at);
    const T* b = row_b(at);
    const int lead = lead_of(a), chunks = (p.vocab + lead + kVerifyChunk - 1) / kVerifyChunk;
    const int c_hi = chunks * (rank + 1) / ranks;
    // The first lane whose running sum passes tau; run becomes the sum before it.
    auto passes = [&](long long mine, int& who) -> bool {
      long long x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x += z;
      }
      const unsigned hit = __ballot_sync(kAll, run + x > tau);
      who = hit ? __ffs(hit) - 1 : 31;
      run += __shfl_sync(kAll, hit ? x - mine : x, who);
      return hit != 0;
    };
    int c = c_lo, who = 0;
    while (!passes(c + lane < c_hi ? chunk_sum[c + lane - c_lo] : 0, who) && c + 32 < c_hi) c += 32;
    c += who;
    // Lane i takes entries 16 i .. 16 i + 15 of the chunk.
    const float cm = (float)C, cl = (float)(C - (double)cm);
    const int y0 = c * kVerifyChunk - lead + lane * kMine;
    int hi[kMine], lo[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int y = y0 + i;
      hi[i] = lo[i] = 0;
      if (y < 0 || y >= p.vocab) continue;
      const float pp = prob(a[y]);
      if (!DRAFT || C == 0.0) add_weight<kVerifyPlain>(pp, 0.f, 0.f, 0.f, hi[i], lo[i]);
      else if (C == 1.0) add_weight<kVerifyOne>(pp, prob(b[y]), cm, cl, hi[i], lo[i]);
      else add_weight<kVerifyMore>(pp, prob(b[y]), cm, cl, hi[i], lo[i]);
    }
    if (take_out)
      for (int j = at + 1; j < n; ++j) {
        if (parent[j] != at) continue;
        const int x = tok[j] - y0;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (x == i) hi[i] = lo[i] = 0;
      }
    long long mine = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) mine += joined(hi[i], lo[i]);
    if (passes(mine, who) && lane == who) {
      int y = y0;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {  // the first entry that passes
        run += joined(hi[i], lo[i]);
        y += run <= tau;
      }
      p.next_tokens[seq] = y;
    }
  }
  if (rank == 0) {
    if (tid == 0) {
      p.path_lens[seq] = len;
      if (all <= 0) {  // a row without any probability
        p.next_tokens[seq] = -1;
        record_error(p.status, PA_ERR_ARG);
      }
    }
    for (int k = len + tid; k < p.max_path_len; k += kVerifyThreads) path[k] = -1;
  }
}

template <typename T>
static cudaError_t launch_verify(const VerifyParams& p, int num_seqs, cudaStream_t stream) {
  // CTAs of a sequence: as many as keep the batch within three per SM and leave
  // each at least four chunks. A sequence's passes get shorter with each (8
  // trees over 131072 fp32 tokens: 67, 41, 28, 22 us with 1, 2, 4, 8), until
  // the batch fills the machine (96 trees: 62, 49, 59 us with 2, 4, 8; 64 over
  // 32000: 23, 23, 33).
  int ranks = 1;
  while (ranks < kVerifyMaxCluster && (int64_t)num_seqs * ranks * 2 <= 3 * num_sms_current_device() &&
         p.vocab / kVerifyChunk >= ranks * 2 * 4)
    ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_seqs * ranks));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.draft ? cudaLaunchKernelEx(&cfg, verify_kernel<T, true>, p)
                 : cudaLaunchKernelEx(&cfg, verify_kernel<T, false>, p);
}

}  // namespace pa

extern "C" int pa_verify_tree(const void* target_probs, int64_t target_stride, const void* draft_probs,
                              int64_t draft_stride, const int32_t* draft_tokens, const int32_t* cu_q_lens,
                              const int32_t* parents, const float* uniform_accept, const float* uniform_sample,
                              int32_t num_seqs, int32_t total_q, int32_t max_q_len, int32_t vocab_size,
                              int32_t max_path_len, int32_t* path, int32_t* path_lens, int32_t* next_tokens,
                              pa_dtype dtype, void* stream) {
  using namespace pa;
  if (num_seqs < 0 || total_q < 0 || vocab_size < 1 || max_path_len < 1) return PA_ERR_ARG;
  if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (vocab_size > kVerifyMaxVocab) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (max_q_len < 0) return PA_ERR_ARG;
  if (max_q_len > kVerifyMaxNodes) return PA_ERR_UNSUPPORTED;
  if (target_stride < vocab_size || (draft_probs && draft_stride < vocab_size)) return PA_ERR_ARG;
  if (!cu_q_lens || !path || !path_lens || !next_tokens) return PA_ERR_ARG;
  const uintptr_t odd = reinterpret_cast<uintptr_t>(target_probs) | reinterpret_cast<uintptr_t>(draft_probs);
  if (odd & (dtype == PA_F32 ? 3u : 1u)) return PA_ERR_ALIGN;
  if (total_q > 0 && (!target_probs || !draft_tokens || !parents || !uniform_accept || !uniform_sample))
    return PA_ERR_ARG;
  int* st = device_status_ptr();
  if (!st) return PA_ERR_CUDA;
  VerifyParams p{};
  p.target = target_probs;
  p.draft = draft_probs;
  p.tokens = draft_tokens;
  p.cu_q_lens = cu_q_lens;
  p.parents = parents;
  p.u_accept = uniform_accept;
  p.u_sample = uniform_sample;
  p.target_stride = target_stride;
  p.draft_stride = draft_stride;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.vocab = vocab_size;
  p.max_path_len = max_path_len;
  p.path = path;
  p.path_lens = path_lens;
  p.next_tokens = next_tokens;
  p.status = st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == PA_F32   ? launch_verify<float>(p, num_seqs, s)
                        : dtype == PA_F16 ? launch_verify<__half>(p, num_seqs, s)
                                          : launch_verify<__nv_bfloat16>(p, num_seqs, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
