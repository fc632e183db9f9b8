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
// order of the sum, so sums are taken over integers: a weight in [0, 1] is
// rounded once to a multiple of 2^-44 (2^18 of them fit 62 bits), and integer
// sums do not depend on their order. p - C q is formed in pairs of floats
// (exact product, exact difference), since double arithmetic runs at a
// fraction of the rate.
//
// A sequence is one cluster of 1 to 8 CTAs, each with a slice of the
// vocabulary; all of them walk the tree by themselves and exchange only sums.
// A warp sums chunks of 512 entries (16 bytes a load, a chunk's loads all in
// flight) and every chunk's sum is kept, so the entry where the running sum
// passes the threshold takes a second look at one chunk only. What bounds it
// is the rows' one pass from HBM; with few sequences, the latency of its
// dependent loads and cluster barriers.
#include <cooperative_groups.h>

#include <algorithm>

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
constexpr double kVerifyUnit = 1.0 / 17592186044416.0;  // 2^-44
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

// max(0, p - C q) in units of 2^-44, as hi * 2^22 + lo with 0 <= hi <= 2^22 and
// |lo| <= 2^21. C = c + cl (cl: what a float of C leaves over).
template <int MODE>
__device__ __forceinline__ void weight_parts(float p, float q, float c, float cl, uint32_t& hi, int& lo) {
  float d = p, e = 0.f;  // p - C q = d + e
  if constexpr (MODE != kVerifyPlain) {
    float m = q, me = 0.f;  // C q = m + me
    if constexpr (MODE == kVerifyMore) {
      m = c * q;
      me = fmaf(cl, q, fmaf(c, q, -m));
    }
    d = p - m;
    const float bb = d - p;
    e = (p - (d - bb)) - (m + bb);
    if constexpr (MODE == kVerifyMore) e -= me;
  }
  const float magic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
  const float t = fmaf(d, 4194304.f, magic);
  float rest = fmaf(d, 4194304.f, magic - t);
  if constexpr (MODE != kVerifyPlain) rest = fmaf(e, 4194304.f, rest);
  const bool some = MODE == kVerifyPlain || d + e > 0.f;
  hi = some ? __float_as_uint(t) - __float_as_uint(magic) : 0u;
  lo = some ? __float2int_rn(rest * 4194304.f) : 0;
}

__device__ __forceinline__ long long joined(uint32_t hi, int lo) { return ((long long)hi << 22) + lo; }

template <typename T>
__device__ __forceinline__ float entry(const uint4& raw, int i) {
  return prob(reinterpret_cast<const T*>(&raw)[i]);
}

// The 16 bytes of a row of V that hold entries y .. of it; entries outside
// the row come as 0. `line`: the address of entry y is a multiple of 16.
template <typename T>
__device__ __forceinline__ uint4 load_line(const T* row, int y, int V, bool line) {
  constexpr int N = 16 / sizeof(T);
  if (line && y >= 0 && y + N <= V) return __ldg(reinterpret_cast<const uint4*>(row + y));
  uint4 raw = make_uint4(0, 0, 0, 0);
  T* t = reinterpret_cast<T*>(&raw);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (y + i >= 0 && y + i < V) t[i] = row[y + i];
  return raw;
}

// A lane's weights of one chunk, at(u, i, hi, lo) for each: entry (32 u +
// lane) N + i of the chunk. y: the row's entry that the lane's first one is.
template <typename T, int MODE, typename F>
__device__ __forceinline__ void chunk_weights(const T* a, const T* b, int y, int V, float c, float cl, F at) {
  constexpr int N = 16 / sizeof(T), kLoads = kVerifyChunk / (32 * N);
  const bool line = ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
  uint4 x[kLoads], z[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    x[u] = load_line(a, y + u * 32 * N, V, true);
    if constexpr (MODE != kVerifyPlain) z[u] = load_line(b, y + u * 32 * N, V, line);
  }
#pragma unroll
  for (int u = 0; u < kLoads; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t hi;
      int lo;
      float q = 0.f;
      if constexpr (MODE != kVerifyPlain) q = entry<T>(z[u], i);
      weight_parts<MODE>(entry<T>(x[u], i), q, c, cl, hi, lo);
      at(u, i, hi, lo);
    }
}

// The sums of a slice's chunks, one warp a chunk at a time; returns this
// warp's share of their total.
template <typename T, int MODE>
__device__ __forceinline__ long long slice_sums(const T* a, const T* b, int lead, int V, float c, float cl, int c_lo,
                                                int c_hi, long long* chunk_sum) {
  constexpr int N = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  long long mine = 0;
#pragma unroll 1
  for (int k = c_lo + (threadIdx.x >> 5); k < c_hi; k += kVerifyWarps) {
    uint32_t h = 0;
    int l = 0;
    chunk_weights<T, MODE>(a, b, k * kVerifyChunk - lead + lane * N, V, c, cl, [&](int, int, uint32_t hi, int lo) {
      h += hi;
      l += lo;
    });
    // 512 entries: at most 2^31, and 2^30 either way.
    const long long s = joined(__reduce_add_sync(kAll, h), __reduce_add_sync(kAll, l));
    if (lane == 0) chunk_sum[k - c_lo] = s;
    mine += s;
  }
  return mine;
}

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads, sizeof(T) == 2 ? 4 : 3) verify_kernel(const VerifyParams p) {
  constexpr int N = 16 / sizeof(T);                // entries of one load
  constexpr int kLoads = kVerifyChunk / (32 * N);  // loads of a lane in a chunk
  constexpr int kMine = kLoads * N;                // entries of a lane in a chunk
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
      if (tid == 0 && n64 != 0) record_error(p.status, bad_len ? PA_ERR_SEQLEN : PA_ERR_ARG);
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
        uint32_t hi;
        int lo;
        weight_parts<kVerifyPlain>(px[j], 0.f, 0.f, 0.f, hi, lo);
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
          if (stale) S = (double)total(at, C, false) * kVerifyUnit;
          const double w = fmax(0.0, (double)px[j] - C * (double)qx[j]);
          if ((double)ua[j] * (double)qx[j] * S < w) {
            step = j;
            break;
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
    uint32_t hi[kMine];
    int lo[kMine];
    const float cm = (float)C, cl = (float)(C - (double)cm);
    const int y0 = c * kVerifyChunk - lead + lane * N;
    auto keep = [&](int u, int i, uint32_t h, int l) { hi[u * N + i] = h, lo[u * N + i] = l; };
    if (C == 0.0) chunk_weights<T, kVerifyPlain>(a, a, y0, p.vocab, cm, cl, keep);
    else chunk_weights<T, DRAFT ? kVerifyMore : kVerifyPlain>(a, b, y0, p.vocab, cm, cl, keep);
    if (take_out)
      for (int j = at + 1; j < n; ++j) {
        if (parent[j] != at) continue;
        const int x = tok[j] + lead - c * kVerifyChunk;  // place in the chunk
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (x == (i / N * 32 + lane) * N + i % N) hi[i] = 0, lo[i] = 0;
      }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      long long mine = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) mine += joined(hi[u * N + i], lo[u * N + i]);
      if (passes(mine, who)) {
        if (lane == who) {
          int y = c * kVerifyChunk - lead + (u * 32 + lane) * N;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const long long w = joined(hi[u * N + i], lo[u * N + i]);
            if (run + w > tau) {
              p.next_tokens[seq] = y + i;
              break;
            }
            run += w;
          }
        }
        break;
      }
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
  // CTAs of a sequence: as many as keep the batch within four per SM and
  // leave each at least four chunks.
  int ranks = 1;
  while (ranks < kVerifyMaxCluster && (int64_t)num_seqs * ranks * 2 <= 4 * num_sms_current_device() &&
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
