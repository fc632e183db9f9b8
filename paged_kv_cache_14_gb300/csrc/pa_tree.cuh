// Tree attention over the paged cache: parameters and the work split shared
// by the tensor-core and the fp32 kernel.
//
// A unit is one (sequence, KV head, query tile): the tile's rows are (tree
// node, query head of the group) pairs and its keys are the sequence's
// ctx + nodes cached positions, cut into key tiles. The units of a batch,
// sequence-major, form one line of key tiles, and CTA b of N takes the tiles
// [W b / N, W (b + 1) / N) of it, so every CTA has the same work (to one
// tile) whatever the lengths are. A CTA writes the units that lie wholly in
// its range; of a unit that crosses a range border every CTA writes its
// (m, l, o~) partial, and a second kernel joins them in CTA order. A CTA has
// at most two such pieces: slot 2b holds the piece of a unit begun by an
// earlier CTA, slot 2b + 1 that of a unit begun here. So the partials need
// 2 N tiles whatever the batch is, and there is no plan kernel: every CTA
// finds its place with a scan of the lengths.
//
// Where trees fill more than one query tile, the tiles of one KV head read
// the same keys. One after another they would read them from HBM again (304
// CTAs' keys do not stay in L2: 2.4 TB read per TB of keys), so CTAs then work
// in teams of two on the line: a place on it is two query tiles of one KV head,
// member r taking the tile 2 i + r, and an odd last tile's place is two KV
// heads (so there are teams only where the number of KV heads is even). The
// members run side by side, and the second read of a key tile finds it in L2
// (1.38 TB read; 48 sequences of 8192 with trees of 40: 403 us without teams,
// 316 with them).
#pragma once

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kMaxTreeNodes = 1024;

// Written by every CTA: the unit it began and did not finish.
struct TreeMerge {
  int32_t parts;   // pieces of the unit (0: nothing to join here)
  int32_t q0;      // first row of the sequence in q / out
  int32_t nodes;
  int32_t kvh;
  int32_t qt;
  int32_t pad[3];
};
static_assert(sizeof(TreeMerge) == 32, "laid out in the workspace");

struct TreeParams {
  const void* q;
  void* out;
  const void* k_cache;
  const void* v_cache;
  const float* kv_scales;  // 8-bit cache: (K, V) scale per (block, KV head); else nullptr
  int32_t kv_fmt;
  const int32_t* block_tables;
  const int32_t* cu_q_lens;
  const int32_t* parents;
  const int32_t* ctx_lens;
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t total_q;
  int32_t max_q_len;
  int32_t max_kv_len;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t num_blocks;
  int32_t group;
  int32_t tile_rows;  // rows of a query tile in use: a multiple of the group, or any number (fp32)
  int32_t tile_m;     // rows of a partial tile in the workspace
  int32_t tile_keys;
  int32_t team;       // CTAs that share a place on the line: 1 or 2
  // A key tile's time in pieces of the join: splitting a unit of n tiles into
  // pieces of t costs t * piece_cost + n / t, so a CTA takes at least
  // sqrt(n / piece_cost) tiles.
  int32_t piece_cost;
  float scale_log2;
  TreeMerge* merge;   // [ctas]
  float* part_o;      // [2 * ctas][tile_m][head_dim]
  float* part_ml;     // [2 * ctas][tile_m][2]
  int* status;
};

// Work of one sequence: key tiles, query tiles and places (units of a team);
// none for an empty or illegal one.
struct TreeSeq {
  int q0, nodes, ctx, ktiles, qtiles, places;
  __device__ __forceinline__ int64_t tiles() const { return (int64_t)ktiles * places; }
};

// Lengths as they stand in memory (sequence i < num_seqs).
struct TreeLens {
  int q0, q1, ctx;
};

__device__ __forceinline__ TreeLens tree_lens(const TreeParams& p, int i) {
  return {__ldg(p.cu_q_lens + i), __ldg(p.cu_q_lens + i + 1), __ldg(p.ctx_lens + i)};
}

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, const TreeLens& r, bool report = false) {
  TreeSeq s;
  s.q0 = r.q0;
  s.ctx = r.ctx;
  s.nodes = s.ktiles = s.qtiles = s.places = 0;
  const int64_t n = (int64_t)r.q1 - r.q0, kv = r.ctx + n;
  // (A sequence without nodes sits the step out, whatever its context is.)
  if (n < 0 || r.q0 < 0 || r.q1 > p.total_q ||
      (n > 0 && (n > p.max_q_len || r.ctx < 0 ||
                 kv > min((int64_t)p.max_kv_len, (int64_t)p.max_blocks_per_seq * p.block_size)))) {
    if (report) record_error(p.status, PA_ERR_SEQLEN);
    return s;
  }
  if (n == 0) return s;
  s.nodes = (int)n;
  s.ktiles = (int)(((uint32_t)kv + p.tile_keys - 1) / (uint32_t)p.tile_keys);
  s.qtiles = (s.nodes * p.group + p.tile_rows - 1) / p.tile_rows;
  s.places = (s.qtiles * p.num_kv_heads) >> (p.team - 1);
  return s;
}

// A team's place on the line of tiles.
struct TreeRange {
  int64_t begin;  // first tile of this team
  int64_t left;   // tiles of this team
  int64_t total;  // tiles of the batch
  int teams;      // teams that share it
  int team;       // this CTA's
  int seq;        // sequence that holds the first tile, and the tile's place in it
  int64_t off;
};

// The scan: threads 0 .. THREADS-1 of the CTA (all of them) sum the tiles of
// a run of sequences each; the one whose run holds the CTA's first tile
// walks it. `sm` is THREADS / 16 + 2 words of 8 bytes.
template <int THREADS>
__device__ __forceinline__ TreeRange tree_range(const TreeParams& p, int64_t* sm) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int per = (p.num_seqs + THREADS - 1) / THREADS;
  const int s0 = min(p.num_seqs, (int)threadIdx.x * per), s1 = min(p.num_seqs, s0 + per);
  int64_t mine = 0, my_units = 0;
  for (int s = s0; s < s1; ++s) {
    const TreeSeq q = tree_seq(p, tree_lens(p, s), blockIdx.x == 0);
    mine += q.tiles();
    my_units += q.places;
  }
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) my_units += __shfl_xor_sync(0xffffffffu, my_units, o);
  if (lane == 31) sm[w] = x, sm[THREADS / 32 + w] = my_units;
  __syncthreads();
  int64_t base = x - mine, total = 0, units = 0;
  for (int i = 0; i < THREADS / 32; ++i) {
    const int64_t t = sm[i];
    if (i < w) base += t;
    total += t;
    units += sm[THREADS / 32 + i];
  }
  TreeRange r;
  r.total = total;
  const float least = sqrtf((float)total / ((float)max(units, (int64_t)1) * p.piece_cost));
  const int64_t most = (int64_t)((float)total / fmaxf(1.f, least));
  r.teams = (int)max((int64_t)1, min((int64_t)(gridDim.x / p.team), most));
  r.team = blockIdx.x / p.team;
  r.begin = 0;
  r.left = 0;
  r.seq = 0;
  r.off = 0;
  if (r.team < r.teams) {
    r.begin = total * r.team / r.teams;
    r.left = total * (r.team + 1) / r.teams - r.begin;
  }
  int64_t* found = sm + THREADS / 16;
  if (r.left > 0 && r.begin >= base && r.begin < base + mine) {
    int64_t at = base;
    for (int s = s0; s < s1; ++s) {
      const int64_t t = tree_seq(p, tree_lens(p, s)).tiles();
      if (r.begin < at + t) {
        found[0] = s;
        found[1] = r.begin - at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  if (r.left > 0) {
    r.seq = (int)found[0];
    r.off = found[1];
  }
  return r;
}

// One piece of a unit: key tiles [t0, t1) of its ktiles.
struct TreePiece {
  TreeSeq s;
  int seq, kvh, qt, t0, t1;
  int64_t at;  // place of tile t0 on the line
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == s.ktiles; }
  __device__ __forceinline__ int kv_len() const { return s.ctx + s.nodes; }
};

// Walks the pieces of a CTA's range. Every role of a CTA runs its own copy, at
// the very point where its pipeline is empty, so a step is kept short: the
// next sequence's lengths are loaded a sequence ahead, and only the first
// piece takes a 64-bit division.
struct TreeWalk {
  TreeSeq s;
  TreeLens ahead;
  int seq, place, t;
  int64_t at, left;
  __device__ __forceinline__ TreeWalk(const TreeParams& p, const TreeRange& r)
      : seq(r.seq), place(0), t(0), at(r.begin), left(r.left) {
    if (left > 0) {
      s = tree_seq(p, tree_lens(p, seq));
      place = (int)(r.off / s.ktiles);
      t = (int)(r.off - (int64_t)place * s.ktiles);
      look(p);
    }
  }
  __device__ __forceinline__ void look(const TreeParams& p) { ahead = tree_lens(p, min(seq + 1, p.num_seqs - 1)); }
  __device__ __forceinline__ bool next(const TreeParams& p, TreePiece& c) {
    if (left <= 0) return false;
    while (place >= s.places) {  // also steps over sequences without work
      ++seq;
      place = 0;
      s = tree_seq(p, ahead);
      look(p);
    }
    c.s = s;
    c.seq = seq;
    c.t0 = t;
    c.t1 = (int)min((int64_t)s.ktiles, t + left);
    if (p.team == 1) {
      c.kvh = place / s.qtiles;
      c.qt = place - c.kvh * s.qtiles;
    } else {
      const int r = blockIdx.x & 1, pairs = s.qtiles >> 1;
      if (place < pairs * p.num_kv_heads) {
        c.kvh = place / pairs;
        c.qt = 2 * (place - c.kvh * pairs) + r;
      } else {
        c.kvh = 2 * (place - pairs * p.num_kv_heads) + r;
        c.qt = s.qtiles - 1;
      }
    }
    c.at = at;
    at += c.t1 - c.t0;
    left -= c.t1 - c.t0;
    ++place;  // (a piece that ends before its unit does is the last one)
    t = 0;
    return true;
  }
};

// Slot of a piece's partial, and what the join kernel needs of a unit begun here.
__device__ __forceinline__ int tree_slot(const TreePiece& c) { return 2 * blockIdx.x + (c.t0 == 0 ? 1 : 0); }

__device__ __forceinline__ void tree_note_merge(const TreeParams& p, const TreeRange& r, const TreePiece& c) {
  // Team of tile w: the b with floor(W b / N) <= w, the largest such b.
  const int64_t last = c.at - c.t0 + c.s.ktiles - 1;
  const int64_t e = ((last + 1) * r.teams - 1) / r.total;
  TreeMerge m;
  m.parts = (int)(e - r.team + 1);
  m.q0 = c.s.q0;
  m.nodes = c.s.nodes;
  m.kvh = c.kvh;
  m.qt = c.qt;
  m.pad[0] = m.pad[1] = m.pad[2] = 0;
  p.merge[blockIdx.x] = m;
}

// Bits of the 32 nodes from `first` on that are `node` or its ancestors.
// parents: the sequence's. A parent that is not below its node ends the walk
// (reported by tree_check_parents).
__device__ __forceinline__ uint32_t tree_ancestors(const int32_t* parents, int node, int first) {
  uint32_t bits = 0;
  while (node >= first && node >= 0) {
    if (node < first + 32) bits |= 1u << (node - first);
    const int up = __ldg(parents + node);
    if (up >= node) break;
    node = up;
  }
  return bits;
}

// Reports parents that are not below their node, once per sequence: by the
// CTA with the last key tile of its first unit.
template <int THREADS>
__device__ __forceinline__ void tree_check_parents(const TreeParams& p, const TreePiece& c, int tid) {
  if (c.kvh || c.qt || c.t1 != c.s.ktiles) return;
  for (int j = tid; j < c.s.nodes; j += THREADS) {
    const int up = __ldg(p.parents + c.s.q0 + j);
    if (up < -1 || up >= j) record_error(p.status, PA_ERR_ARG);
  }
}

// The tensor-core kernel (fp16 / bf16 q; head_dim 64 or 128, 128 for 8-bit
// caches): query tiles of 128 rows, key tiles of 64 positions.
constexpr int kTreeTcRows = 128;
constexpr int kTreeTcKeys = 64;
int launch_tree_tc(const TreeParams& p, int ctas, pa_dtype dt, cudaStream_t stream);

}  // namespace pa
