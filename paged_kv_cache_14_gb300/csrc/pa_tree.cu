// Tree attention over the paged cache: entry points, the CUDA-core kernel
// and the kernel that joins the pieces of a unit.
//
// One pass of a draft tree: node j of a sequence (its K/V cached at position
// ctx + j) attends to the ctx committed positions and to itself and its
// ancestors in the tree:
//   out[j] = sum_t exp(s_t - max s) v_t / sum_t exp(s_t - max s),
//   s_t = scale q[j] . k_t,  t in {0 .. ctx-1} and {ctx + a : a = j or above j}.
#include <math_constants.h>

#include <algorithm>
#include <cmath>

#include "pa_tree.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// CUDA-core kernel (fp32 I/O): exact fp32 arithmetic. 128 threads, a query tile of 32
// rows (row = node * group + head), key tiles of 32 positions in
// shared memory. Threads 4r .. 4r+3 own row r: eight scores each (keys
// i, i + 4, ...), then every fourth group of four columns of the output.
// ---------------------------------------------------------------------------
namespace ts {
constexpr int kRows = 32;
constexpr int kKeys = 32;
constexpr int kThreads = 128;
constexpr int kPs = kKeys + 4;  // row stride of the weights
__host__ __device__ constexpr int smem_bytes(int d) {
  return (kRows * (d + 4) + kKeys * (d + 4) + kKeys * d + kRows * kPs) * 4;
}
}  // namespace ts

template <int D>
__global__ void __launch_bounds__(ts::kThreads) tree_simt_kernel(const TreeParams p) {
  using namespace ts;
  extern __shared__ float4 smem4[];
  float* qs = reinterpret_cast<float*>(smem4);  // [kRows][D + 4]
  float* ks = qs + kRows * (D + 4);             // [kKeys][D + 4]
  float* vs = ks + kKeys * (D + 4);             // [kKeys][D]
  float* ps = vs + kKeys * D;                   // [kRows][kPs]
  __shared__ int64_t scan[kThreads / 32 + 4];
  __shared__ int blk[kKeys / 16];

  pdl_trigger();
  const TreeRange range = tree_range<kThreads>(p, scan);
  if (threadIdx.x == 0) p.merge[blockIdx.x].parts = 0;
  const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
  TreeWalk walk(range);
  TreePiece c;
  while (walk.next(p, c)) {
    const int32_t* parents = p.parents + c.s.q0;
    tree_check_parents<kThreads>(p, c, threadIdx.x);
    const int32_t* table = p.block_tables + (int64_t)c.seq * p.max_blocks_per_seq;
    const int rows = c.s.nodes * p.group;
    const int r = c.qt * kRows + row;  // row of the unit
    const int node = min(r / p.group, c.s.nodes - 1);
    const int kv_len = c.kv_len();
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
      const int rr = i / (D / 4), d4 = (i - rr * (D / 4)) * 4;
      const int ur = c.qt * kRows + rr;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ur < rows) {
        const int nd = ur / p.group, h = c.kvh * p.group + ur - nd * p.group;
        x = __ldg(reinterpret_cast<const float4*>(
            static_cast<const float*>(p.q) + ((int64_t)(c.s.q0 + nd) * p.num_q_heads + h) * D + d4));
      }
      *reinterpret_cast<float4*>(qs + rr * (D + 4) + d4) = x;
    }
    float m = -CUDART_INF_F, l = 0.f;
    float4 o[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = c.t0; t < c.t1; ++t) {
      const int k0 = t * kKeys;
      __syncthreads();  // the previous tile (or piece) is read
      if (threadIdx.x < kKeys / 16) {
        const int pos = k0 + threadIdx.x * 16;
        int id = -1;
        if (pos < kv_len) {
          id = table[pos / p.block_size];
          if (id < 0 || id >= p.num_blocks) {
            record_error(p.status, PA_ERR_BLOCK_OOB);
            id = -1;
          }
        }
        blk[threadIdx.x] = id;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < kKeys * (D / 4); i += kThreads) {
        const int key = i / (D / 4), d4 = (i - key * (D / 4)) * 4;
        const int id = blk[key / 16];
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (id >= 0 && k0 + key < kv_len) {
          const int64_t tile = (int64_t)id * p.num_kv_heads + c.kvh;
          const int64_t at = (tile * p.block_size + (k0 + key) % p.block_size) * D + d4;
          k = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.k_cache) + at));
          v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.v_cache) + at));
        }
        *reinterpret_cast<float4*>(ks + key * (D + 4) + d4) = k;
        *reinterpret_cast<float4*>(vs + key * D + d4) = v;
      }
      __syncthreads();
      // Keys that this row sees, one bit each.
      uint32_t seen = 0xffffffffu;
      if (k0 + kKeys > c.s.ctx) {
        const int first = k0 - c.s.ctx;  // node of the tile's first key (below 0: context)
        seen = tree_ancestors(parents, node, first);
        if (first < 0) seen |= (1u << (-first)) - 1u;
      }
      float s[kKeys / 4];
#pragma unroll
      for (int j = 0; j < kKeys / 4; ++j) s[j] = 0.f;
      for (int d = 0; d < D; d += 4) {
        const float4 qv = *reinterpret_cast<const float4*>(qs + row * (D + 4) + d);
#pragma unroll
        for (int j = 0; j < kKeys / 4; ++j) {
          const float4 kv = *reinterpret_cast<const float4*>(ks + (part + 4 * j) * (D + 4) + d);
          s[j] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[j]))));
        }
      }
      float mx = m;
#pragma unroll
      for (int j = 0; j < kKeys / 4; ++j) {
        s[j] = (seen >> (part + 4 * j)) & 1u ? s[j] * p.scale_log2 : -CUDART_INF_F;
        mx = fmaxf(mx, s[j]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // A row that has seen no key yet keeps m = -inf and l = 0.
      const float ref = mx == -CUDART_INF_F ? 0.f : mx;
      const float alpha = exp2f(m - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kKeys / 4; ++j) {
        const float w = exp2f(s[j] - ref);
        sum += w;
        ps[row * kPs + part + 4 * j] = w;
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      l = l * alpha + sum;
      m = mx;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[j].x *= alpha, o[j].y *= alpha, o[j].z *= alpha, o[j].w *= alpha;
      for (int key = 0; key < kKeys; ++key) {
        // Values behind the mask may hold anything: they are left out, not
        // multiplied by 0.
        if (!((seen >> key) & 1u)) continue;
        const float w = ps[row * kPs + key];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(vs + key * D + (part + 4 * j) * 4);
          o[j].x = fmaf(w, v.x, o[j].x);
          o[j].y = fmaf(w, v.y, o[j].y);
          o[j].z = fmaf(w, v.z, o[j].z);
          o[j].w = fmaf(w, v.w, o[j].w);
        }
      }
    }
    __syncthreads();
    if (c.whole()) {
      if (r < rows) {
        const float inv = 1.f / l;
        const int h = c.kvh * p.group + r - node * p.group;
        float* out = static_cast<float*>(p.out) + ((int64_t)(c.s.q0 + node) * p.num_q_heads + h) * D;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          store4(out + (part + 4 * j) * 4, make_float4(o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv));
      }
    } else {
      if (c.t0 == 0 && threadIdx.x == 0) tree_note_merge(p, range, c);
      const int64_t slot = (int64_t)tree_slot(c) * kRows + row;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        __stcg(reinterpret_cast<float4*>(p.part_o + slot * D + (part + 4 * j) * 4), o[j]);
      if (part == 0) __stcg(reinterpret_cast<float2*>(p.part_ml + slot * 2), make_float2(m, l));
    }
  }
}

// ---------------------------------------------------------------------------
// Join: block (b, y) joins rows of the unit that CTA b began and did not
// finish. m in log2 units: out = sum_i 2^(m_i - M) o~_i / sum_i 2^(m_i - M) l_i.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeParams p) {
  pdl_wait();
  const TreeMerge mg = p.merge[blockIdx.x];
  if (mg.parts == 0) return;
  const int D = p.head_dim, d4s = D / 4;
  const int rows = min(p.tile_rows, mg.nodes * p.group - mg.qt * p.tile_rows);
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < rows * d4s; i += gridDim.y * kJoinThreads) {
    const int r = i / d4s, d4 = (i - r * d4s) * 4;
    auto slot = [&](int k) -> int64_t {
      return (int64_t)(2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * p.tile_m + r;
    };
    float M = -CUDART_INF_F;
    for (int k = 0; k < mg.parts; ++k) M = fmaxf(M, __ldcg(p.part_ml + slot(k) * 2));
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < mg.parts; ++k) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + slot(k) * 2));
      if (ml.x == -CUDART_INF_F && ml.y == 0.f) continue;  // the row sees none of this piece's keys
      const float w = exp2f(ml.x - M);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + slot(k) * D + d4));
      L = fmaf(w, ml.y, L);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
    const float inv = 1.f / L;
    const int ur = mg.qt * p.tile_rows + r;
    const int node = ur / p.group, h = mg.kvh * p.group + ur - node * p.group;
    store4(static_cast<T*>(p.out) + ((int64_t)(mg.q0 + node) * p.num_q_heads + h) * D + d4,
           make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
}

template <int D>
static int run_simt(const TreeParams& p, int ctas, cudaStream_t stream) {
  auto kern = tree_simt_kernel<D>;
  constexpr int smem = ts::smem_bytes(D);
  if (set_max_dynamic_smem(reinterpret_cast<const void*>(kern), smem) != PA_OK) return PA_ERR_CUDA;
  kern<<<ctas, ts::kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

static int launch_tree_simt(const TreeParams& p, int ctas, cudaStream_t stream) {
  switch (p.head_dim) {
    case 32: return run_simt<32>(p, ctas, stream);
    case 64: return run_simt<64>(p, ctas, stream);
    case 96: return run_simt<96>(p, ctas, stream);
    case 128: return run_simt<128>(p, ctas, stream);
    case 160: return run_simt<160>(p, ctas, stream);
    case 192: return run_simt<192>(p, ctas, stream);
    case 224: return run_simt<224>(p, ctas, stream);
    case 256: return run_simt<256>(p, ctas, stream);
  }
  return PA_ERR_UNSUPPORTED;
}

static int launch_tree_join(const TreeParams& p, int ctas, pa_dtype dt, cudaStream_t stream) {
  const int chunks = std::max(1, (p.tile_m * p.head_dim / 4) / kJoinThreads);
  const dim3 grid(ctas, chunks), block(kJoinThreads);
  cudaError_t e;
  if (dt == PA_F32) e = launch_dependent(tree_join_kernel<float>, grid, block, 0, stream, p);
  else if (dt == PA_F16) e = launch_dependent(tree_join_kernel<__half>, grid, block, 0, stream, p);
  else e = launch_dependent(tree_join_kernel<__nv_bfloat16>, grid, block, 0, stream, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

namespace {

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

// Tiles, grid and workspace of a call; what the size query and the launch share.
struct TreeLayout {
  int rc = PA_OK;
  int ctas = 0, tile_rows = 0, tile_m = 0, tile_keys = 0, min_tiles = 1;
  size_t merge = 0, part_o = 0, part_ml = 0, total = 0;
};

TreeLayout tree_layout(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                       int32_t block_size, int32_t total_q, int32_t max_q_len, int32_t max_kv_len, pa_dtype dt) {
  TreeLayout w;
  auto fail = [&](int rc) {
    w.rc = rc;
    return w;
  };
  if (num_seqs < 0 || total_q < 0 || head_dim < 1 || num_q_heads < 1 || num_kv_heads < 1) return fail(PA_ERR_ARG);
  if (num_q_heads % num_kv_heads) return fail(PA_ERR_HEADS);
  if (block_size != 16 && block_size != 32) return fail(PA_ERR_BLOCKSIZE);
  if (dt != PA_F32 && dt != PA_F16 && dt != PA_BF16) return fail(PA_ERR_DTYPE);
  const int group = num_q_heads / num_kv_heads;
  if (dt == PA_F32) {
    if (head_dim < 32 || head_dim > 256 || head_dim % 32) return fail(PA_ERR_UNSUPPORTED);
  } else if ((head_dim != 64 && head_dim != 128) || group > 128) {
    return fail(PA_ERR_UNSUPPORTED);
  }
  if (num_seqs == 0 || total_q == 0) return w;
  if (max_q_len < 1 || max_kv_len < 1) return fail(PA_ERR_ARG);
  if (num_seqs > 65535 || max_q_len > kMaxTreeNodes) return fail(PA_ERR_UNSUPPORTED);
  int per_sm;
  if (dt == PA_F32) {
    w.tile_rows = w.tile_m = ts::kRows;
    w.tile_keys = ts::kKeys;
    w.min_tiles = 4;
    per_sm = head_dim <= 128 ? 4 : 2;
  } else {
    w.tile_m = kTreeTcRows;
    w.tile_rows = kTreeTcRows / group * group;
    w.tile_keys = kTreeTcKeys;
    w.min_tiles = 2;
    per_sm = 2;
  }
  // Most key tiles there can be: one more query tile than its rows fill for every sequence.
  const double units = ((double)total_q * group / w.tile_rows + std::min(num_seqs, total_q)) * num_kv_heads;
  const double most = units * ((max_kv_len + w.tile_keys - 1) / w.tile_keys) / w.min_tiles + 1;
  w.ctas = (int)std::max(1.0, std::min(most, (double)per_sm * num_sms_current_device()));
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  w.part_o = up((size_t)w.ctas * sizeof(TreeMerge));
  w.part_ml = up(w.part_o + (size_t)2 * w.ctas * w.tile_m * head_dim * 4);
  w.total = up(w.part_ml + (size_t)2 * w.ctas * w.tile_m * 2 * 4);
  return w;
}

int decode_tree(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents, const void* k_cache,
                const void* v_cache, const float* kv_scales, int32_t kv_fmt, const int32_t* block_tables,
                int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len,
                int32_t max_kv_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                int32_t num_blocks, float scale, void* out, void* workspace, size_t workspace_bytes, pa_dtype dtype,
                bool kv8, cudaStream_t stream) {
  const TreeLayout w = tree_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, total_q, max_q_len,
                                   max_kv_len, dtype);
  if (w.rc != PA_OK) return w.rc;
  if (max_blocks_per_seq < 1 || num_blocks < 1 || !std::isfinite(scale)) return PA_ERR_ARG;
  if (dtype != PA_F32 && !(scale > 0.f)) return PA_ERR_ARG;
  if (kv8 && dtype == PA_F32) return PA_ERR_DTYPE;
  if (kv8 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_blocks * num_kv_heads * block_size >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  if (!q || !cu_q_lens || !parents || !k_cache || !v_cache || !block_tables || !ctx_lens || !out) return PA_ERR_ARG;
  if (kv8 && !kv_scales) return PA_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(kv_scales))
    return PA_ERR_ALIGN;
  if (!workspace || workspace_bytes < w.total) return PA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PA_ERR_ALIGN;
  int* st = device_status_ptr();
  if (!st) return PA_ERR_CUDA;
  TreeParams p{};
  p.q = q;
  p.out = out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_scales = kv_scales;
  p.kv_fmt = kv_fmt;
  p.block_tables = block_tables;
  p.cu_q_lens = cu_q_lens;
  p.parents = parents;
  p.ctx_lens = ctx_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.max_kv_len = max_kv_len;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.group = num_q_heads / num_kv_heads;
  p.tile_rows = w.tile_rows;
  p.tile_m = w.tile_m;
  p.tile_keys = w.tile_keys;
  p.min_tiles = w.min_tiles;
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.merge = reinterpret_cast<TreeMerge*>(ws + w.merge);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  p.status = st;
  const int rc = dtype == PA_F32 ? launch_tree_simt(p, w.ctas, stream) : launch_tree_tc(p, w.ctas, dtype, stream);
  if (rc != PA_OK) return rc;
  return launch_tree_join(p, w.ctas, dtype, stream);
}
}  // namespace
}  // namespace pa

extern "C" {

size_t pa_decode_tree_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t block_size, int32_t total_q, int32_t max_q_len, int32_t max_kv_len,
                                     pa_dtype dtype) {
  const pa::TreeLayout w = pa::tree_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, total_q,
                                           max_q_len, max_kv_len, dtype);
  return w.rc == PA_OK ? w.total : 0;
}

int pa_decode_tree(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                   const void* k_cache, const void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                   const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len, int32_t max_kv_len,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t num_blocks, float scale, void* out, void* workspace, size_t workspace_bytes,
                   pa_dtype dtype, void* stream) {
  return pa::decode_tree(q, total_q, cu_q_lens, parents, k_cache, v_cache, nullptr, 0, block_tables,
                         max_blocks_per_seq, ctx_lens, num_seqs, max_q_len, max_kv_len, num_q_heads, num_kv_heads,
                         head_dim, block_size, num_blocks, scale, out, workspace, workspace_bytes, dtype, false,
                         static_cast<cudaStream_t>(stream));
}

int pa_decode_tree_fp8(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                       const void* k_cache, const void* v_cache, const float* kv_scales, const int32_t* block_tables,
                       int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len,
                       int32_t max_kv_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                       int32_t block_size, int32_t num_blocks, float scale, void* out, void* workspace,
                       size_t workspace_bytes, pa_dtype dtype, void* stream) {
  return pa::decode_tree(q, total_q, cu_q_lens, parents, k_cache, v_cache, kv_scales, pa::PA_KV_E4M3, block_tables,
                         max_blocks_per_seq, ctx_lens, num_seqs, max_q_len, max_kv_len, num_q_heads, num_kv_heads,
                         head_dim, block_size, num_blocks, scale, out, workspace, workspace_bytes, dtype, true,
                         static_cast<cudaStream_t>(stream));
}

int pa_decode_tree_e5m2(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                        const void* k_cache, const void* v_cache, const float* kv_scales,
                        const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                        int32_t num_seqs, int32_t max_q_len, int32_t max_kv_len, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                        void* out, void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream) {
  return pa::decode_tree(q, total_q, cu_q_lens, parents, k_cache, v_cache, kv_scales, pa::PA_KV_E5M2, block_tables,
                         max_blocks_per_seq, ctx_lens, num_seqs, max_q_len, max_kv_len, num_q_heads, num_kv_heads,
                         head_dim, block_size, num_blocks, scale, out, workspace, workspace_bytes, dtype, true,
                         static_cast<cudaStream_t>(stream));
}

}  // extern "C"
