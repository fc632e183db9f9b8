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
// rounded once to a multiple of 2^-45 (below 2^18 of them fit 64 bits), and
// integer sums do not depend on their order.
#include <algorithm>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kVerifyMaxNodes = 1024;
constexpr int kVerifyMaxVocab = 1 << 18;
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

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

// max(0, p - C q) as a multiple of 2^-45.
__device__ __forceinline__ long long weight_fixed(float p, float q, double C) {
  const double w = (double)p - C * (double)q;
  return w > 0.0 ? __double2ll_rn(w * 35184372088832.0) : 0ll;
}

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p) {
  __shared__ int16_t parent[kVerifyMaxNodes];
  __shared__ int tok[kVerifyMaxNodes];
  __shared__ float px[kVerifyMaxNodes], qx[kVerifyMaxNodes], ua[kVerifyMaxNodes];
  __shared__ long long wsum[kVerifyWarps];
  __shared__ int bad, state[4];
  __shared__ double mult;
  const int seq = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* path = p.path + (int64_t)seq * p.max_path_len;
  const int q0 = p.cu_q_lens[seq];
  const int64_t n64 = (int64_t)p.cu_q_lens[seq + 1] - q0;
  if (tid == 0) bad = n64 < 0 || q0 < 0 || q0 + n64 > p.total_q || n64 > p.max_q_len;
  __syncthreads();
  const int n = bad ? 0 : (int)n64;
  for (int j = tid; j < n; j += kVerifyThreads) {
    const int up = p.parents[q0 + j];
    parent[j] = (int16_t)up;
    if (up < -1 || up >= j || (j == 0 && up != -1)) bad = 1;
    const int t = p.tokens[q0 + j];
    const bool real = t >= 0 && t < p.vocab && up >= 0 && up < j;
    tok[j] = real ? t : -1;
    ua[j] = p.u_accept[q0 + j];
    px[j] = real ? prob(static_cast<const T*>(p.target)[(int64_t)(q0 + up) * p.target_stride + t]) : 0.f;
    qx[j] = real && DRAFT ? prob(static_cast<const T*>(p.draft)[(int64_t)(q0 + up) * p.draft_stride + t]) : 0.f;
  }
  __syncthreads();
  if (bad || n == 0) {
    if (tid == 0 && bad) record_error(p.status, n64 < 0 || n64 > p.max_q_len || q0 < 0 || q0 + n64 > p.total_q ? PA_ERR_SEQLEN : PA_ERR_ARG);
    for (int k = tid; k < p.max_path_len; k += kVerifyThreads) path[k] = -1;
    if (tid == 0) p.path_lens[seq] = 0, p.next_tokens[seq] = -1;
    return;
  }
  auto row_p = [&](int r) { return static_cast<const T*>(p.target) + (int64_t)(q0 + r) * p.target_stride; };
  auto row_q = [&](int r) { return static_cast<const T*>(p.draft) + (int64_t)(q0 + r) * p.draft_stride; };
  // Warp w sums entries [w seg, (w + 1) seg).
  const int seg = (p.vocab + kVerifyWarps - 1) / kVerifyWarps;
  const int v0 = min(p.vocab, warp * seg), v1 = min(p.vocab, v0 + seg);
  auto total = [&](int r, double C) -> long long {
    const T* a = row_p(r);
    const T* b = DRAFT ? row_q(r) : a;
    long long s = 0;
    for (int y = v0 + lane; y < v1; y += 32) s += weight_fixed(prob(a[y]), DRAFT && C > 0.0 ? prob(b[y]) : 0.f, C);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (lane == 0) wsum[warp] = s;
    __syncthreads();
    long long all = 0;
    for (int i = 0; i < kVerifyWarps; ++i) all += wsum[i];
    return all;
  };

  // The walk. Every thread takes the same steps over shared memory.
  int at = 0, len = 1;
  double C = 0.0;
  if (tid == 0) path[0] = 0;
  while (true) {
    double S = 1.0;
    C = 0.0;
    int step = -1;
    for (int j = at + 1; j < n && len < p.max_path_len; ++j) {
      if (parent[j] != at || tok[j] < 0) continue;
      double w = px[j];
      if constexpr (DRAFT) {
        if (C > 0.0 && S < 0.0) S = (double)total(at, C) * (1.0 / 35184372088832.0);  // put off until a child needs it
        w = fmax(0.0, w - C * (double)qx[j]);
        if ((double)ua[j] * (double)qx[j] * S < w) step = j;
        else if (C == 0.0) C = 1.0, S = -1.0;
        else C += S, S = -1.0;
      } else {
        bool again = false;
        for (int i = at + 1; i < j; ++i) again |= parent[i] == at && tok[i] == tok[j];
        if (again) w = 0.0;
        if ((double)ua[j] * S < w) step = j;
        else S -= w;
      }
      if (step >= 0) break;
    }
    if (step < 0) break;
    at = step;
    if (tid == 0) path[len] = at;
    ++len;
  }
  const bool tried = len < p.max_path_len;  // a full path keeps nothing more: its last node's children are not tried
  // The next token: the weights' sum, then the segment and the entry where
  // the running sum passes u' of it.
  auto gone = [&](int y) {  // without q: y is the token of a refused child
    if (DRAFT || !tried) return false;
    for (int j = at + 1; j < n; ++j)
      if (parent[j] == at && tok[j] == y) return true;
    return false;
  };
  auto dropped = [&](int lo, int hi) -> long long {  // what refused tokens in [lo, hi) take from a sum of p
    long long s = 0;
    if (DRAFT || !tried) return s;
    for (int j = at + 1; j < n; ++j) {
      if (parent[j] != at || tok[j] < lo || tok[j] >= hi) continue;
      bool again = false;
      for (int i = at + 1; i < j; ++i) again |= parent[i] == at && tok[i] == tok[j];
      if (!again) s += weight_fixed(px[j], 0.f, 0.0);
    }
    return s;
  };
  long long all = total(at, C) - dropped(0, p.vocab);
  bool plain = false;
  if (all <= 0) {  // nothing left after the refusals: drawn from the target itself
    C = 0.0;
    plain = true;
    all = total(at, 0.0);
  }
  const float us = fminf(__saturatef(p.u_sample[seq]), 0.99999994f);
  const long long tau = (long long)((double)us * (double)all);
  long long before = 0;
  for (int i = 0; i < warp; ++i)
    before += wsum[i] - (plain ? 0 : dropped(min(p.vocab, i * seg), min(p.vocab, (i + 1) * seg)));
  const long long mine = wsum[warp] - (plain ? 0 : dropped(v0, v1));
  if (all > 0 && before <= tau && tau < before + mine) {
    const T* a = row_p(at);
    const T* b = DRAFT ? row_q(at) : a;
    long long run = before;
    for (int y0 = v0; y0 < v1; y0 += 32) {
      const int y = y0 + lane;
      long long w = 0;
      if (y < v1 && (plain || !gone(y))) w = weight_fixed(prob(a[y]), DRAFT && C > 0.0 ? prob(b[y]) : 0.f, C);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += z;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + w > tau);
      if (hit) {
        if (lane == 0) p.next_tokens[seq] = y0 + __ffs(hit) - 1;
        break;
      }
      run += __shfl_sync(0xffffffffu, w, 31);
    }
  }
  if (tid == 0) {
    p.path_lens[seq] = len;
    if (all <= 0) {  // a row without any probability
      p.next_tokens[seq] = -1;
      record_error(p.status, PA_ERR_ARG);
    }
  }
  for (int k = len + tid; k < p.max_path_len; k += kVerifyThreads) path[k] = -1;
}

template <typename T>
static cudaError_t launch_verify(const VerifyParams& p, int num_seqs, cudaStream_t stream) {
  if (p.draft) verify_kernel<T, true><<<num_seqs, kVerifyThreads, 0, stream>>>(p);
  else verify_kernel<T, false><<<num_seqs, kVerifyThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
