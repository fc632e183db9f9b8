/*
 * libpagedattn — paged KV-cache attention for one NVIDIA GB300 (sm_103a).
 *
 * The KV cache of every sequence lives in fixed-size physical blocks of
 * `block_size` tokens; a per-sequence block table maps logical block
 * floor(pos / block_size) to a physical block id, and the token sits at
 * offset pos mod block_size inside it ("High-Throughput Local LLM
 * Infrastructure: Architecting a Distributed Go API Gateway for vLLM &
 * PagedAttention Clusters", section 1.2 "PagedAttention Mechanics & Virtual
 * Page Tables"; "Inside vLLM: Anatomy of a High-Throughput LLM Inference
 * System (2025)", section "Physical Block Mapping and Kernel Invocation").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All pointers named *_cache, q, k, v, out, block_tables, seq_lens,
 *    ctx_lens, cu_q_lens, slot_mapping, seq_ids, positions and workspace are
 *    DEVICE pointers on the current CUDA device, owned by the caller. The
 *    library allocates nothing and keeps no pointer after a call returns.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 *    legacy default stream). Host-side argument errors return a negative
 *    status BEFORE anything is launched, and then no output is touched.
 *  - Errors found on the device (an out-of-range block id or slot, a
 *    sequence longer than its table or than max_seq_len, a bounded wait that
 *    ran out) never trap: the kernel skips the bad access, records the first
 *    error code in a per-device status word and carries on. pa_get_status()
 *    reads and clears that word. Rows hit by such an error hold unspecified
 *    values.
 *  - Cache layout: k_cache and v_cache are separate pools, each
 *    [num_blocks][num_kv_heads][block_size][head_dim], contiguous, so one
 *    (block, KV head) tile of block_size x head_dim elements is contiguous.
 *  - q, k, v, out and the caches of one call share one dtype (pa_dtype).
 *    Arithmetic is fp32 (scores, softmax, accumulation) whatever the I/O
 *    dtype.
 *  - Grouped-query attention: num_q_heads must be a multiple of
 *    num_kv_heads; query head h reads KV head h / (num_q_heads/num_kv_heads).
 *  - Device pointers to tensors must be 16-byte aligned.
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_dtype {
  PA_F32 = 0,
  PA_F16 = 1,
  PA_BF16 = 2
} pa_dtype;

/* Status codes. 0 is success; every error is negative. */
#define PA_OK 0
#define PA_ERR_ARG (-1)         /* null pointer, negative size, bad stride */
#define PA_ERR_DTYPE (-2)       /* dtype not supported by this entry point  */
#define PA_ERR_HEADS (-3)       /* num_q_heads not a multiple of num_kv_heads */
#define PA_ERR_BLOCKSIZE (-4)   /* block_size must be 16 or 32              */
#define PA_ERR_WORKSPACE (-5)   /* workspace null or smaller than required  */
#define PA_ERR_ALIAS (-6)       /* copy_blocks: dst repeated or also a src  */
#define PA_ERR_BLOCK_OOB (-7)   /* device: block id / slot outside the pool */
#define PA_ERR_SEQLEN (-8)      /* device: length < 1, > table, > max given */
#define PA_ERR_CUDA (-9)        /* a CUDA runtime call failed               */
#define PA_ERR_UNSUPPORTED (-10)/* head_dim (or shape) not supported        */
#define PA_ERR_TIMEOUT (-11)    /* device: a bounded wait ran out           */
#define PA_ERR_ALIGN (-12)      /* a tensor pointer is not 16-byte aligned  */
#define PA_ERR_SCRATCH (-13)    /* pa_decode_noalloc: call needs more scratch than its fixed array */

/* Human-readable name of a status code (static storage). */
const char* pa_strerror(int status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int pa_version(void);

/*
 * pa_get_status — synchronise `stream`, return the first device-side error
 * recorded since the last call (PA_OK if none), and clear it. The status
 * word is per device and shared by all streams. Its device address is looked
 * up once per device and cached for the life of the process, so the library
 * must not be used across a cudaDeviceReset.
 */
int pa_get_status(void* stream);

/*
 * pa_slot_mapping — slot of every new token.
 *   slot_mapping[t] = block_tables[seq_ids[t]][positions[t] / block_size]
 *                     * block_size + positions[t] % block_size
 * (logical block index and block offset of section 1.2 of the "High-
 * Throughput Local LLM Infrastructure" page).
 *   block_tables : int32 [num_seqs][max_blocks_per_seq]
 *   seq_ids      : int32 [num_tokens], 0 <= seq_ids[t] < num_seqs
 *   positions    : int32 [num_tokens], 0 <= positions[t] < max_blocks_per_seq*block_size
 *   slot_mapping : int64 [num_tokens] (output)
 * A token whose seq id, position or physical block (>= num_blocks) is out of
 * range gets slot -1 and PA_ERR_BLOCK_OOB is recorded. num_tokens == 0 is a
 * no-op.
 */
int pa_slot_mapping(const int32_t* block_tables, int32_t max_blocks_per_seq, int32_t num_seqs,
                    const int32_t* seq_ids, const int32_t* positions, int64_t num_tokens,
                    int32_t block_size, int32_t num_blocks, int64_t* slot_mapping, void* stream);

/*
 * pa_reshape_and_cache — scatter new tokens' K and V into their cache slots
 * (section 2.1 "PagedAttention Memory Allocation Life-Cycle", step 4: the
 * kernels write new K/V into the assigned physical blocks).
 *   k, v         : [num_tokens][num_kv_heads][head_dim], contiguous
 *   slot_mapping : int64 [num_tokens]; slot s writes block s / block_size,
 *                  offset s % block_size; s < 0 skips the token (padding);
 *                  s >= num_blocks*block_size records PA_ERR_BLOCK_OOB and
 *                  skips the token
 *   k_cache, v_cache : the pools (layout above), updated in place
 * Bit-exact copy. head_dim * sizeof(dtype) must be a multiple of 16.
 * Two tokens with the same slot race (one of them wins).
 */
int pa_reshape_and_cache(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                         void* k_cache, void* v_cache, int32_t num_blocks, int32_t block_size,
                         int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, void* stream);

/*
 * pa_copy_blocks — copy-on-write copies: for every pair, the whole K block
 * and V block (all KV heads) dst <- src ("High-Throughput Local LLM
 * Infrastructure...", section 1.2, "Reference Counting & Copy-on-Write";
 * "03 - PagedAttention & the vLLM V1 Architecture", section "The block
 * table walkthrough": the whole block is copied when a write inside it would
 * diverge).
 *   src_dst_pairs : HOST int64 [num_pairs][2] (src, dst). The pairs are
 *                   validated on the host before any launch: every id in
 *                   [0, num_blocks) else PA_ERR_BLOCK_OOB; no dst repeated
 *                   and no dst equal to any src, else PA_ERR_ALIAS. They are
 *                   passed to the kernel by value (no device copy), so the
 *                   host array may be reused as soon as the call returns.
 *   block_bytes   : bytes of one block of one pool
 *                   (num_kv_heads*block_size*head_dim*sizeof(dtype)),
 *                   a multiple of 16.
 * Bit-exact. num_pairs == 0 is a no-op.
 */
int pa_copy_blocks(void* k_cache, void* v_cache, const int64_t* src_dst_pairs, int32_t num_pairs,
                   int32_t num_blocks, int64_t block_bytes, void* stream);

/*
 * pa_swap_blocks — swap preemption ("Inside vLLM: Anatomy of a
 * High-Throughput LLM Inference System (2025)", section "Preemption
 * Mechanics: Swapping vs. Recomputation"; "03 - PagedAttention & the vLLM V1
 * Architecture", section "Preemption & eviction": a preempted sequence's
 * blocks are written out to a host pool and later brought back, possibly
 * into other physical blocks). For every pair, the whole block
 * dst_pool[dst] <- src_pool[src] of the K pool and, if given, the V pool.
 *   src_k, src_v : source pools ([src_num_blocks] blocks of block_bytes)
 *   dst_k, dst_v : destination pools ([dst_num_blocks] blocks)
 *                  Each pool is device memory, managed memory or pinned
 *                  (page-locked: cudaHostAlloc / cudaHostRegister) host
 *                  memory; the kernel reads and writes host memory directly
 *                  (over NVLink-C2C on Grace-Blackwell). Pageable host memory
 *                  returns PA_ERR_ARG. src_v and dst_v are both NULL (one
 *                  pool, e.g. the scales of an e4m3 cache) or both given.
 *   src_dst_pairs : HOST int64 [num_pairs][2] (src, dst), validated before
 *                  any launch: src in [0, src_num_blocks), dst in
 *                  [0, dst_num_blocks) else PA_ERR_BLOCK_OOB; no dst repeated
 *                  and, when src and dst are the same pool, no dst equal to a
 *                  src, else PA_ERR_ALIAS. Passed to the kernel by value.
 *   block_bytes  : bytes of one block of one pool, a multiple of 4
 *                  (PA_ERR_UNSUPPORTED otherwise); 16-byte vectors are used
 *                  when it is a multiple of 16 and the pools are aligned.
 * Bit-exact. num_pairs == 0 is a no-op.
 */
int pa_swap_blocks(const void* src_k, const void* src_v, void* dst_k, void* dst_v, const int64_t* src_dst_pairs,
                   int32_t num_pairs, int32_t src_num_blocks, int32_t dst_num_blocks, int64_t block_bytes,
                   void* stream);

/*
 * Split-KV partitioning of decode. A sequence of L keys is cut into
 * ceil(L / partition_size) partitions; each is reduced to (m, l, o~)
 * partials (running max, sum of exp(s - m), unnormalised output) in the
 * workspace, and a second pass merges them:
 *   out = sum_p exp(m_p - M) o~_p / sum_p exp(m_p - M) l_p,  M = max_p m_p.
 * A sequence with one partition is written directly. partition_size must be
 * a positive multiple of block_size, or 0 for the library's choice, which
 * depends on (num_seqs, num_kv_heads, num_q_heads, block_size, max_seq_len)
 * and the current device's SM count.
 *
 * pa_decode_partition_size returns the partition size a call with these
 * arguments uses (resolving 0), or a negative status.
 * pa_decode_workspace_size returns the workspace bytes pa_decode needs for
 * these arguments: a work list (about num_seqs*max_parts*4 bytes) plus,
 * when a sequence can need
 * more than one partition, fp32 partials of
 * num_seqs*num_q_heads*max_parts*(head_dim+2)*4 bytes, with
 * max_parts = ceil(max_seq_len / partition_size). It is never 0 for a
 * non-empty batch.
 */
int32_t pa_decode_partition_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t block_size, int32_t max_seq_len, int32_t partition_size);
size_t pa_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t block_size, int32_t max_seq_len,
                                int32_t partition_size);

/*
 * pa_decode — paged decode attention, one new query token per sequence
 * ("03 - PagedAttention & the vLLM V1 Architecture", section "The attention
 * kernel side": walk the block table, fetch each block's K and V tiles,
 * compute softmax(Q K^T / sqrt(d)) V over the gathered tiles; the attention
 * equation of "Inside vLLM...", section "Physical Block Mapping and Kernel
 * Invocation").
 *   q            : [num_seqs][num_q_heads][head_dim]
 *   block_tables : int32 [num_seqs][max_blocks_per_seq]
 *   seq_lens     : int32 [num_seqs]; sequence i attends to keys
 *                  0 .. seq_lens[i]-1 (its newest token included: cache it
 *                  with pa_reshape_and_cache first)
 *   max_seq_len  : an upper bound of seq_lens (host value; sizes the grid);
 *                  a longer sequence records PA_ERR_SEQLEN
 *   scale        : multiplies q.k (usually 1/sqrt(head_dim))
 *   out          : [num_seqs][num_q_heads][head_dim]
 *   workspace    : device scratch of pa_decode_workspace_size() bytes,
 *                  16-byte aligned; contents need no initialisation (every
 *                  call rewrites what it uses). Two calls whose executions
 *                  overlap on the device (different streams) must not share
 *                  a workspace.
 * Supported: block_size 16 or 32; fp16/bf16 with head_dim 64 or 128 (tensor-
 * core path); fp32 with head_dim a multiple of 32 up to 256 (CUDA-core
 * path). Each KV block is read once per KV head: all query heads of a GQA
 * group are processed together.
 */
int pa_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
              int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
              int32_t num_blocks, float scale, void* out, int32_t partition_size, void* workspace,
              size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * pa_decode_shared_prefix — pa_decode for batches in which groups of
 * consecutive sequences share leading KV blocks through their block tables
 * (prefix caching or parallel sampling: several tables name the same
 * refcounted physical blocks, "High-Throughput Local LLM Infrastructure...",
 * section 1.2 "Reference Counting & Copy-on-Write"; "Inside vLLM...",
 * section "Zero-Copy Branching and Parallel Sampling"). The result is the
 * same attention as pa_decode; what changes is the work: each group's shared
 * blocks are read once per KV head for all its members, in one tcgen05
 * tensor-core pass whose rows are (member, query head), and each member's
 * private suffix goes through the split-KV decode kernel; the two are merged
 * with log-sum-exp weights.
 *   group_starts : int32 [num_groups+1] device; group g is the sequences
 *                  group_starts[g] .. group_starts[g+1]-1 (consecutive;
 *                  group_starts[0] = 0, group_starts[num_groups] = num_seqs)
 *   prefix_lens  : int32 [num_seqs] device; a hint: sequence i shares its
 *                  first prefix_lens[i] tokens with its group. A hint is used
 *                  only if it is a positive multiple of block_size, shorter
 *                  than seq_lens[i], and the first prefix_lens[i]/block_size
 *                  table entries of sequence i equal those of the group member
 *                  with the longest hint; otherwise it is ignored for that
 *                  sequence (same result, no saving). Malformed group_starts
 *                  record PA_ERR_ARG and disable every hint.
 *   workspace    : pa_decode_shared_prefix_workspace_size() bytes.
 * Other arguments as pa_decode. fp16/bf16, head_dim 64 or 128, GQA group G of at
 * most 128 (2 * floor(128 / G) members per tensor-core work item, in two
 * tiles; larger groups take several items), scale > 0.
 */
size_t pa_decode_shared_prefix_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t block_size, int32_t max_seq_len,
                                              int32_t partition_size, int32_t num_groups);
int pa_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                            int32_t max_seq_len, const int32_t* group_starts, const int32_t* prefix_lens,
                            int32_t num_groups, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            int32_t block_size, int32_t num_blocks, float scale, void* out, int32_t partition_size,
                            void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * pa_decode_step — one decode step in a single call: the same work and
 * results as pa_copy_blocks, pa_slot_mapping, pa_reshape_and_cache and
 * pa_decode, in that order. The decode plan (it reads only block_tables
 * and seq_lens, which the other three do not write) is launched first and
 * the copies, slots and cache write run beside it; the decode kernel starts
 * once the cache write has completed. Arguments as pa_decode_step_shared_prefix
 * without the sharing groups; the workspace is pa_decode_workspace_size()
 * bytes. fp16/bf16 only (PA_ERR_DTYPE otherwise). Every host check runs
 * before the first launch.
 */
int pa_decode_step(const int64_t* cow_pairs, int32_t num_cow_pairs, const int32_t* new_seq_ids,
                   const int32_t* new_positions, const void* k_new, const void* v_new, int64_t num_new_tokens,
                   int64_t* slot_mapping, const void* q, void* k_cache, void* v_cache, const int32_t* block_tables,
                   int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t num_blocks, float scale, void* out, int32_t partition_size, void* workspace,
                   size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * pa_decode_step_shared_prefix — one decode step of a prefix-sharing batch
 * in a single call: the same work and results as, in this order,
 *   pa_copy_blocks(k_cache, v_cache, cow_pairs, num_cow_pairs, ...),
 *   pa_slot_mapping(block_tables, ..., new_seq_ids, new_positions,
 *                   num_new_tokens, ..., slot_mapping),
 *   pa_reshape_and_cache(k_new, v_new, slot_mapping, num_new_tokens, ...),
 *   pa_decode_shared_prefix(q, k_cache, v_cache, block_tables, ...)
 * (a serving step: copy-on-write of shared blocks about to be written,
 * "High-Throughput Local LLM Infrastructure...", section 1.2; slots and the
 * cache write of the step's new tokens, section 1.2 and "Inside vLLM...",
 * "PagedAttention"; then the attention of the new query tokens).
 * Because every kernel of the step is this library's, the call launches the
 * shared-prefix check first and runs the copies, slots and cache write beside
 * it (it reads only block_tables, seq_lens, group_starts and prefix_lens,
 * which they do not write); the attention kernels start once the cache write
 * has completed.
 *   cow_pairs      : int64 [num_cow_pairs][2] HOST (src, dst) block ids, as
 *                    pa_copy_blocks (may be NULL when num_cow_pairs == 0)
 *   new_seq_ids, new_positions : int32 [num_new_tokens] device, as
 *                    pa_slot_mapping
 *   k_new, v_new   : [num_new_tokens][num_kv_heads][head_dim] device, dtype
 *   slot_mapping   : int64 [num_new_tokens] device, written
 * Other arguments as pa_decode_shared_prefix. Every host check of the four
 * calls runs before the first launch: a rejected call launches nothing.
 * fp16/bf16 only (PA_ERR_DTYPE otherwise). Errors as the four calls.
 */
int pa_decode_step_shared_prefix(const int64_t* cow_pairs, int32_t num_cow_pairs, const int32_t* new_seq_ids,
                                 const int32_t* new_positions, const void* k_new, const void* v_new,
                                 int64_t num_new_tokens, int64_t* slot_mapping, const void* q, void* k_cache,
                                 void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                                 const int32_t* group_starts, const int32_t* prefix_lens, int32_t num_groups,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                 int32_t num_blocks, float scale, void* out, int32_t partition_size, void* workspace,
                                 size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * pa_decode_noalloc — pa_decode for callers that cannot allocate device
 * memory when they call (for example a plugin running inside another
 * runtime's fixed memory pool, a serving loop that forbids cudaMalloc after
 * start-up because it synchronises the device, or code that must not create
 * allocations while a stream is being captured). The pages describe no such
 * call; it exists for these callers only.
 * Same arguments, checks and results as pa_decode, without workspace
 * arguments: the split-KV scratch is a fixed device array of
 * pa_decode_noalloc_scratch_limit() bytes (64 MiB) inside the library, held
 * on a device until the process exits once the library's code is loaded
 * there. The call itself calls no cudaMalloc, cudaFree or allocating
 * library routine. A call whose pa_decode_workspace_size() exceeds the limit
 * returns PA_ERR_SCRATCH before launching anything.
 * The first call on a device looks up the array's device address (with that
 * device current) and caches it. Under CUDA's default lazy module loading
 * that lookup is what loads the library's module on the device, so the first
 * call makes a one-time 64 MiB device reservation and may synchronise: make
 * it during set-up, before any stream capture and before the point after
 * which the caller may not allocate. All calls share the one array and it
 * keeps the last call's contents (nothing in it needs to start at zero): two
 * calls whose executions overlap on the device, on different streams, race
 * on it. The cached address is that of the device's primary context: do not
 * use the library across a cudaDeviceReset.
 */
size_t pa_decode_noalloc_scratch_limit(void);
int pa_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                      int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                      int32_t num_blocks, float scale, void* out, int32_t partition_size, pa_dtype dtype,
                      void* stream);

/*
 * pa_chunked_prefill — attention of a mixed batch (prefill chunks and
 * decode rows) over the paged context (chunked prefill: "Tech Radar: vLLM v1
 * Production Engine Architecture...", section 3 "Dynamic Chunked Prefill").
 *   q          : [total_q][num_q_heads][head_dim]; sequence i owns rows
 *                cu_q_lens[i] .. cu_q_lens[i+1]-1
 *   cu_q_lens  : int32 [num_seqs+1], cu_q_lens[0] = 0, non-decreasing,
 *                cu_q_lens[num_seqs] = total_q
 *   ctx_lens   : int32 [num_seqs]; tokens before sequence i's chunk. Row r
 *                of the chunk sits at position ctx_lens[i] + r and attends to
 *                keys 0 .. ctx_lens[i] + r (causal inside the chunk). The
 *                chunk's own K/V must already be cached (pa_reshape_and_cache
 *                of its tokens first).
 *   max_q_len, max_kv_len : host upper bounds of the q_len and of
 *                ctx_len + q_len over the batch; a sequence above them
 *                records PA_ERR_SEQLEN and is skipped
 *   out        : [total_q][num_q_heads][head_dim]
 *   workspace  : pa_chunked_prefill_workspace_size() bytes, 16-byte aligned,
 *                no initialisation needed; not shared by overlapping calls
 * Rows with q_len == 1 go through the decode path (any supported dtype and
 * head_dim). Longer chunks in fp16/bf16 go through a tcgen05 tensor-core
 * kernel that needs head_dim 64 or 128, a GQA group G of at most 128 (a
 * tensor-core tile holds floor(128 / G) query positions x G heads)
 * (PA_ERR_UNSUPPORTED otherwise) and scale > 0 (PA_ERR_ARG); fp32 chunks go
 * through a CUDA-core kernel with exact fp32 arithmetic (head_dim as for
 * fp32 decode, any scale), one query row at a time: exact, not fast.
 * Precondition of the tensor-core kernel, not checked by this version: one
 * chunk holds at most 65536 work items of two tiles, i.e. max_q_len <=
 * 65536 * 2 * floor(128 / G) (131072 rows at G = 128, 2097152 at G = 8);
 * rows of a longer chunk past that bound are not computed.
 */
size_t pa_chunked_prefill_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t block_size, int32_t total_q,
                                         int32_t max_kv_len);
int pa_chunked_prefill(const void* q, int32_t total_q, const int32_t* cu_q_lens, const void* k_cache,
                       const void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                       const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len, int32_t max_kv_len,
                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                       int32_t num_blocks, float scale, void* out, void* workspace, size_t workspace_bytes,
                       pa_dtype dtype, void* stream);

/*
 * FP8 (e4m3) KV cache with per-block scales ("Tech Radar: vLLM v1 Production
 * Engine Architecture...", section 2, "Hopper TMA Warp Specialization & FP8
 * Kernel Integration", item 3 "FP8 Block-Quantized Caching": keys and values
 * are quantized dynamically to 8-bit floating point at block boundaries,
 * halving the bytes per token; "High-Throughput Local LLM Infrastructure...",
 * section 6, Q5: e4m3).
 *   k_cache, v_cache : uint8 pools [num_blocks][num_kv_heads][block_size][head_dim]
 *                      of e4m3 codes (OCP FP8 E4M3: bias 7, no infinity,
 *                      largest finite 448)
 *   kv_scales        : float32 [num_blocks][num_kv_heads][2], 16-byte aligned:
 *                      the K (index 0) and V (index 1) scale of every (block,
 *                      KV head) tile. Stored value = e4m3 value * scale.
 * Scale rule of a cache write, per (block, KV head, pool), with a = the
 * largest |x| the call writes into the block and o_min the lowest offset it
 * writes there: s_old = 0 if o_min == 0 (the write starts the block afresh),
 * else the stored scale; s_new = max(s_old, fl32(a / 448)); if s_new > s_old
 * > 0 the codes at offsets < o_min are re-encoded as e4m3(fl32(value *
 * fl32(s_old / s_new))); each new row is encoded as e4m3(fl32(x / s_new))
 * (code 0 when s_new == 0). e4m3() rounds to nearest, ties to even, and
 * saturates at +-448. Codes at offsets above the written ones are untouched.
 */

/*
 * pa_reshape_and_cache_fp8 — cache write into the e4m3 pools.
 *   k, v         : [num_tokens][num_kv_heads][head_dim] of dtype (fp32, fp16
 *                  or bf16), 16-byte aligned
 *   slot_mapping : int64 [num_tokens], as for pa_reshape_and_cache. All the
 *                  tokens a call writes into one block must be consecutive
 *                  entries of slot_mapping (entries with slot < 0 may sit
 *                  between them): the order in which a batch lists each
 *                  sequence's new tokens. Tokens of one block split into two
 *                  separate runs race on that block's codes and scale (the
 *                  result is unspecified; nothing outside the block is
 *                  touched).
 * head_dim must be 64 or 128 (PA_ERR_UNSUPPORTED). Bit-exact (see the rule
 * above). Two tokens with the same slot: the later one in the list wins.
 */
int pa_reshape_and_cache_fp8(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                             void* k_cache, void* v_cache, float* kv_scales, int32_t num_blocks, int32_t block_size,
                             int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, void* stream);

/*
 * pa_copy_blocks_fp8 — copy-on-write for the e4m3 pools: for every pair the
 * whole K and V block and the block's 2 * num_kv_heads scales, dst <- src.
 * Pairs are validated as for pa_copy_blocks (HOST array, PA_ERR_BLOCK_OOB,
 * PA_ERR_ALIAS). Bit-exact.
 */
int pa_copy_blocks_fp8(void* k_cache, void* v_cache, float* kv_scales, const int64_t* src_dst_pairs,
                       int32_t num_pairs, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                       int32_t head_dim, void* stream);

/*
 * pa_decode_fp8 — pa_decode over the e4m3 pools: every stored value is the
 * e4m3 code times its (block, KV head) scale, and the attention is that of
 * pa_decode on those values. q and out are fp16 or bf16 (dtype;
 * PA_ERR_DTYPE otherwise); head_dim must be 128 (PA_ERR_UNSUPPORTED). The
 * workspace is pa_decode_workspace_size() bytes, as for pa_decode. Codes are
 * widened to fp16 exactly; scores, softmax and accumulation are fp32.
 */
int pa_decode_fp8(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                  const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                  int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                  int32_t block_size, int32_t num_blocks, float scale, void* out, int32_t partition_size,
                  void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * pa_decode_shared_prefix_fp8 — pa_decode_shared_prefix over the e4m3 pools:
 * the attention of pa_decode_fp8 (every stored value is the e4m3 code times
 * its (block, KV head) scale), computed as pa_decode_shared_prefix computes
 * it: each group's shared blocks once per KV head for all its members in the
 * tcgen05 tensor-core pass, the private suffixes in the split-KV decode, the
 * two merged with log-sum-exp weights. FP8 block-quantised caching is the
 * page's pairing for serving many concurrent 70B-class sequences ("Tech
 * Radar: vLLM v1 Production Engine Architecture...", section 2, item 3;
 * "High-Throughput Local LLM Infrastructure...", section 6, Q5); prefix
 * sharing is section 1.2 of the latter, "Reference Counting &
 * Copy-on-Write".
 *   k_cache, v_cache, kv_scales : the e4m3 pools and scales, as for
 *                  pa_decode_fp8 (kv_scales 16-byte aligned, else PA_ERR_ALIGN;
 *                  NULL with num_seqs > 0: PA_ERR_ARG)
 * Other arguments, hints, checks and errors as pa_decode_shared_prefix; the
 * workspace is pa_decode_shared_prefix_workspace_size() bytes. q/out fp16
 * or bf16, head_dim 128, GQA group up to 128, scale > 0.
 * The codes are widened to fp16 exactly (a bf16 query row is moved into fp16
 * by a power of two); scores, softmax and accumulation are fp32.
 */
int pa_decode_shared_prefix_fp8(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                                const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                int32_t num_seqs, int32_t max_seq_len, const int32_t* group_starts,
                                const int32_t* prefix_lens, int32_t num_groups, int32_t num_q_heads,
                                int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                float scale, void* out, int32_t partition_size, void* workspace,
                                size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * pa_chunked_prefill_fp8 — pa_chunked_prefill over the e4m3 pools (chunked
 * prefill mixed with decode rows, "Tech Radar...", section 3 "Dynamic
 * Chunked Prefill", over the FP8 block-quantised cache of section 2, item
 * 3): the attention of pa_chunked_prefill on the dequantised values. Decode
 * rows go through the e4m3 decode kernel, chunks through the tcgen05 kernel
 * with the codes widened to fp16 in shared memory. Arguments as
 * pa_chunked_prefill plus kv_scales (as pa_decode_fp8); the workspace is
 * pa_chunked_prefill_workspace_size() bytes. q/out fp16 or bf16 (else
 * PA_ERR_DTYPE), head_dim 128 (else PA_ERR_UNSUPPORTED); chunks need a
 * GQA group up to 128 and scale > 0.
 */
int pa_chunked_prefill_fp8(const void* q, int32_t total_q, const int32_t* cu_q_lens, const void* k_cache,
                           const void* v_cache, const float* kv_scales, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len,
                           int32_t max_kv_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t block_size, int32_t num_blocks, float scale, void* out, void* workspace,
                           size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * e5m2 KV cache: the other 8-bit format the page names for block-quantised
 * caching ("Tech Radar: vLLM v1 Production Engine Architecture...", section
 * 2, "Hopper TMA Warp Specialization & FP8 Kernel Integration", item 3:
 * e4m3 or e5m2). Same pools, scales, scale rule and errors as the e4m3 calls
 * above, with the OCP FP8 E5M2 codec in place of e4m3:
 *   k_cache, v_cache : uint8 pools [num_blocks][num_kv_heads][block_size][head_dim]
 *                      of e5m2 codes (sign, 5 exponent bits with bias 15, 2
 *                      mantissa bits; exponent field 31 holds infinities and
 *                      NaNs; largest finite 57344)
 *   kv_scales        : float32 [num_blocks][num_kv_heads][2], as above
 * The cache write's scale is s_new = max(s_old, fl32(a / 57344)) and every
 * code is e5m2(fl32(x / s)) (round to nearest even, saturating at +-57344,
 * so the cache only ever writes finite codes); re-encoding on scale growth
 * as for e4m3. The attention calls widen every code to fp16 exactly (an
 * e5m2 code is the upper byte of the fp16 of the same value). Codes past a
 * sequence's end may hold any bits, infinities and NaNs included.
 * pa_copy_blocks_fp8 copies e5m2 pools and their scales unchanged (it moves
 * bytes and scales, whatever the format).
 */

/* pa_reshape_and_cache_e5m2 — pa_reshape_and_cache_fp8 writing e5m2 codes. */
int pa_reshape_and_cache_e5m2(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                              void* k_cache, void* v_cache, float* kv_scales, int32_t num_blocks, int32_t block_size,
                              int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, void* stream);

/* pa_decode_e5m2 — pa_decode_fp8 over e5m2 pools (same arguments). */
int pa_decode_e5m2(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                   const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                   int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                   int32_t block_size, int32_t num_blocks, float scale, void* out, int32_t partition_size,
                   void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream);

/* pa_decode_shared_prefix_e5m2 — pa_decode_shared_prefix_fp8 over e5m2 pools
 * (same arguments, hints, checks and workspace). */
int pa_decode_shared_prefix_e5m2(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                 int32_t num_seqs, int32_t max_seq_len, const int32_t* group_starts,
                                 const int32_t* prefix_lens, int32_t num_groups, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                 float scale, void* out, int32_t partition_size, void* workspace,
                                 size_t workspace_bytes, pa_dtype dtype, void* stream);

/* pa_chunked_prefill_e5m2 — pa_chunked_prefill_fp8 over e5m2 pools (same
 * arguments and workspace). */
int pa_chunked_prefill_e5m2(const void* q, int32_t total_q, const int32_t* cu_q_lens, const void* k_cache,
                            const void* v_cache, const float* kv_scales, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len,
                            int32_t max_kv_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            int32_t block_size, int32_t num_blocks, float scale, void* out, void* workspace,
                            size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * Draft trees (speculative decoding). A step offers every sequence a tree of
 * drafted tokens instead of one new token ("Speculative decoding": Medusa,
 * EAGLE and n-gram drafts, in the vLLM architecture page's section on V1
 * features); the target scores the whole tree at once, the drafts that agree
 * with it are kept, and their K/V rows stay in the cache. The three calls
 * below are one step's: write the nodes' K/V with pa_reshape_and_cache (or
 * its 8-bit forms) at positions ctx .. ctx + nodes - 1, attend with
 * pa_decode_tree in every layer, choose with pa_verify_tree, and move the
 * kept rows together with pa_compact_tree.
 *
 * Trees are given as parents, ragged over the batch:
 *   cu_q_lens : int32 [num_seqs+1]; sequence i owns the nodes (rows of q, of
 *               the probabilities, ...) cu_q_lens[i] .. cu_q_lens[i+1]-1; none
 *               is allowed (a sequence that sits the step out)
 *   parents   : int32 [total_q]; the parent of each node as a node number
 *               within its sequence, lower than the node's own; -1 for a
 *               root. Node 0 is the newest committed token.
 * A sequence has at most max_q_len nodes, and max_q_len at most 1024
 * (PA_ERR_UNSUPPORTED).
 */

/*
 * pa_decode_tree - attention of tree nodes over the paged context. Node j of
 * sequence i sits in the cache at position ctx_lens[i] + j and attends to
 * keys 0 .. ctx_lens[i]-1, to itself and to its ancestors, and to nothing
 * else: whatever the K/V rows of other branches or of the positions behind
 * the tree hold (infinities and NaN included) does not reach it. (In an 8-bit
 * pool a block's scale is part of the value of each of its rows.)
 *   q          : [total_q][num_q_heads][head_dim]
 *   ctx_lens   : int32 [num_seqs]; committed tokens before the tree (>= 0)
 *   max_q_len, max_kv_len : host upper bounds of the nodes and of ctx + nodes
 *                of a sequence (no sequence may have more than 2^31 - 64); a
 *                sequence above them, or with a cu_q_lens that falls or leaves
 *                [0, total_q], records PA_ERR_SEQLEN and its rows are not
 *                written
 *   out        : [total_q][num_q_heads][head_dim]; must not overlap q
 *   workspace  : pa_decode_tree_workspace_size() bytes, 16-byte aligned, no
 *                initialisation needed; not shared by calls that overlap. Its
 *                size follows the bounds given (num_seqs, total_q, max_q_len,
 *                max_kv_len), not the lengths, up to what the device's SM
 *                count sets: one made for larger bounds serves smaller ones.
 * A parent that is not below its node records PA_ERR_ARG (the node then
 * counts as a root); a block outside the pool records PA_ERR_BLOCK_OOB, and
 * the rows that see it are unspecified. num_seqs is at most 65535. fp16/bf16:
 * head_dim 64 or 128, a GQA group of at most 128, pools of fewer than 2^31 rows
 * (num_blocks * num_kv_heads * block_size) and scale > 0 (PA_ERR_UNSUPPORTED,
 * PA_ERR_ARG otherwise); the softmax weights are rounded to the 16-bit type
 * (over 8-bit pools to fp16) for the second product, as in pa_decode: a weight
 * is off by half a step of that type, in fp16 by 2^-25 at most below 2^-14.
 * fp32: head_dim a multiple of 32 up to 256, exact fp32 arithmetic, any finite
 * scale. Rows are computed from their own sequence alone; results do not
 * depend on the order in which the device runs.
 */
size_t pa_decode_tree_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t block_size, int32_t total_q, int32_t max_q_len, int32_t max_kv_len,
                                     pa_dtype dtype);
int pa_decode_tree(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                   const void* k_cache, const void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                   const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len, int32_t max_kv_len,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t num_blocks, float scale, void* out, void* workspace, size_t workspace_bytes,
                   pa_dtype dtype, void* stream);

/* pa_decode_tree_fp8, pa_decode_tree_e5m2 - pa_decode_tree over the 8-bit
 * pools (kv_scales as for pa_decode_fp8, 16-byte aligned). q/out fp16 or bf16
 * (else PA_ERR_DTYPE), head_dim 128 (else PA_ERR_UNSUPPORTED). */
int pa_decode_tree_fp8(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                       const void* k_cache, const void* v_cache, const float* kv_scales, const int32_t* block_tables,
                       int32_t max_blocks_per_seq, const int32_t* ctx_lens, int32_t num_seqs, int32_t max_q_len,
                       int32_t max_kv_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                       int32_t block_size, int32_t num_blocks, float scale, void* out, void* workspace,
                       size_t workspace_bytes, pa_dtype dtype, void* stream);
int pa_decode_tree_e5m2(const void* q, int32_t total_q, const int32_t* cu_q_lens, const int32_t* parents,
                        const void* k_cache, const void* v_cache, const float* kv_scales,
                        const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                        int32_t num_seqs, int32_t max_q_len, int32_t max_kv_len, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                        void* out, void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream);

/*
 * pa_verify_tree - which drafted tokens are kept, and the token after them,
 * so that the kept tokens and the next one are distributed as the target
 * alone would draw them (speculative sampling).
 *   target_probs : [total_q][vocab_size] of dtype, rows target_stride elements
 *                  apart; row r: the target's distribution of the token after
 *                  node r
 *   draft_probs  : the same for the draft (draft_stride): row r is the
 *                  distribution that the children of node r were drawn from,
 *                  independently; or NULL: the children were chosen, not
 *                  drawn (a lookup, the likeliest few). Children drawn without
 *                  replacement are neither: the kept tokens would not be
 *                  distributed as the target's.
 *   draft_tokens : int32 [total_q]; the token of each node (a root's is not
 *                  read). A node whose token lies outside [0, vocab_size) is
 *                  padding: never kept.
 *   uniform_accept : float [total_q], uniform_sample : float [num_seqs];
 *                  random numbers in [0, 1), one for each node and sequence
 *   path         : int32 [num_seqs][max_path_len] (output): the kept nodes
 *                  from node 0 down, then -1
 *   path_lens    : int32 [num_seqs] (output): kept nodes; at least 1 (node 0)
 *                  unless the sequence has no nodes
 *   next_tokens  : int32 [num_seqs] (output): the token drawn at the last kept
 *                  node; -1 for a sequence without nodes
 * From node 0 on, the children of the last kept node are tried in node order.
 * With its target row p, draft row q, w = p and S = 1, child c with token x
 * is kept if uniform_accept[c] * q(x) * S < w(x); otherwise w becomes
 * max(0, w - S q) and S the sum of w, and the next child is tried. Without
 * draft_probs child c is kept if uniform_accept[c] * S < w(x); otherwise S
 * drops by w(x) and w(x) becomes 0. Where no child is kept (or the path is
 * full: then none is tried) the next token is the smallest y with
 * w(0) + .. + w(y) > uniform_sample * sum(w); if every w is 0, w = p is used.
 * Probabilities outside [0, 1] are held to it and NaN counts as 0; a row
 * without any probability gives next token -1 and PA_ERR_ARG. Sums are taken
 * over weights formed from whole multiples of 2^-43 (within two of them),
 * exactly, so results do not depend on the order in which the device runs (a
 * mass of w below some 2^-40 is not resolved; refusals leave that little only
 * with that probability). A sequence whose cu_q_lens falls, leaves
 * [0, total_q] or has more than max_q_len nodes records PA_ERR_SEQLEN, one with
 * a parent that is not below its node (or a node 0 that is no root)
 * PA_ERR_ARG; both get path_lens 0 and next token -1. vocab_size is at most
 * 262144 (PA_ERR_UNSUPPORTED), max_path_len at least 1. Rows need no alignment
 * beyond their element's (PA_ERR_ALIGN).
 */
int pa_verify_tree(const void* target_probs, int64_t target_stride, const void* draft_probs, int64_t draft_stride,
                   const int32_t* draft_tokens, const int32_t* cu_q_lens, const int32_t* parents,
                   const float* uniform_accept, const float* uniform_sample, int32_t num_seqs, int32_t total_q,
                   int32_t max_q_len, int32_t vocab_size, int32_t max_path_len, int32_t* path, int32_t* path_lens,
                   int32_t* next_tokens, pa_dtype dtype, void* stream);

/*
 * pa_compact_tree - moves the kept nodes' K/V rows together: in every layer,
 * for k < path_lens[i], the rows of position ctx_lens[i] + path[i][k] go to
 * position ctx_lens[i] + k, as if all were read before any is written. The
 * sequence then has ctx_lens[i] + path_lens[i] cached tokens.
 *   k_caches, v_caches : HOST arrays of num_layers device pointers, the pools
 *                  of each layer (same shape, none twice: PA_ERR_ARG; one
 *                  block table serves them all; layers that share a pool list
 *                  it once); the arrays are read before the call returns
 *   path, path_lens : int32 device, as pa_verify_tree writes them; any
 *                  strictly rising path of nodes >= 0 will do, and length 0.
 *                  max_path_len at most 1024.
 * Bit-exact; every other row stays as it is. The blocks written must be the
 * sequence's own (copy shared ones first). head_dim * sizeof(dtype) must be a
 * multiple of 16, num_kv_heads * head_dim at most 2^20 (PA_ERR_UNSUPPORTED). A sequence with a negative context, a length outside
 * [0, max_path_len] or a position past its block table records
 * PA_ERR_SEQLEN, a path that does not rise PA_ERR_ARG, a block outside the
 * pool PA_ERR_BLOCK_OOB; nothing of it is moved.
 */
int pa_compact_tree(void* const* k_caches, void* const* v_caches, int32_t num_layers, const int32_t* block_tables,
                    int32_t max_blocks_per_seq, const int32_t* ctx_lens, const int32_t* path,
                    const int32_t* path_lens, int32_t num_seqs, int32_t max_path_len, int32_t num_blocks,
                    int32_t block_size, int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, void* stream);

/*
 * pa_compact_tree_fp8, pa_compact_tree_e5m2 - the same over 8-bit pools.
 *   kv_scales : HOST array of num_layers device pointers, float32
 *               [num_blocks][num_kv_heads][2] each
 * Scale rule, per (block, KV head, pool) that rows land in: with o the offset
 * of the first of them, s_new = the largest of the landing rows' scales (their
 * source blocks', before the call) and, if o > 0, the block's own; codes at
 * offsets below o are re-encoded by fl32(s_old / s_new) if s_new > s_old > 0,
 * as a cache write does; a landing row whose scale is s_new keeps its codes,
 * another is encoded as code(fl32(value * fl32(s_source / s_new))). Codes at
 * offsets above the landing rows are untouched (their scale may not be: the
 * rows of dropped nodes hold no meaning any more). head_dim 64 or 128
 * (PA_ERR_UNSUPPORTED).
 */
int pa_compact_tree_fp8(void* const* k_caches, void* const* v_caches, float* const* kv_scales, int32_t num_layers,
                        const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                        const int32_t* path, const int32_t* path_lens, int32_t num_seqs, int32_t max_path_len,
                        int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                        void* stream);
int pa_compact_tree_e5m2(void* const* k_caches, void* const* v_caches, float* const* kv_scales, int32_t num_layers,
                         const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* ctx_lens,
                         const int32_t* path, const int32_t* path_lens, int32_t num_seqs, int32_t max_path_len,
                         int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                         void* stream);

/*
 * Long contexts: a decode step that reads part of the cache. A step rotates
 * its new tokens' queries and keys by their positions and caches them
 * (pa_rope_and_cache), keeps an 8-bit summary of the keys of every block
 * (pa_block_summaries), chooses for every sequence and KV head the blocks
 * whose summaries promise the largest scores (pa_select_blocks), and attends
 * to these (pa_decode_sparse). The block tables are those of section 1.2 of
 * the "High-Throughput Local LLM Infrastructure" page; the chosen blocks are a
 * subset of each table's entries.
 */

/* How pa_rope_table scales the frequencies f_i = base^(-2 i / rot_dim) of the
 * pairs i = 0 .. rot_dim/2 - 1. */
#define PA_ROPE_NONE 0
#define PA_ROPE_LINEAR 1 /* f_i / factor */
#define PA_ROPE_BASE 2   /* base * factor^(rot_dim / (rot_dim - 2)) in base's place */
#define PA_ROPE_BANDS 3  /* by turns: with t = original_len f_i / (2 pi) and
                          * w = (t - low) / (high - low) held to [0, 1],
                          * w f_i + (1 - w) f_i / factor */
#define PA_ROPE_RAMP 4   /* by pair: with d(t) = rot_dim ln(original_len / (2 pi t)) / (2 ln base),
                          * a = max(floor(d(high)), 0), z = min(ceil(d(low)), rot_dim - 1) and
                          * w = (i - a) / max(z - a, 0.001) held to [0, 1],
                          * (1 - w) f_i + w f_i / factor; models with such
                          * frequencies commonly turn with an amplitude of
                          * 0.1 ln(factor) + 1, which the caller passes */

/*
 * pa_rope_table - cosines and sines of positions first_position ..
 * first_position + num_positions - 1:
 *   cos_sin : float [num_positions][rot_dim] (output), 16-byte aligned; row
 *             p holds amplitude cos(a_i) at [i] and amplitude sin(a_i) at
 *             [rot_dim/2 + i], a_i = (first_position + p) f_i
 * Frequencies are computed in twice the doubles' precision and angles reduced
 * in 64-bit fixed point: an entry of amplitude 1 is within 2^-22 of the cosine
 * or sine, at frequencies of up to 2^24 radians a position. Positions lie
 * below 2^31; rot_dim is even, 2 to 256 (PA_ERR_UNSUPPORTED); base > 1, factor
 * > 0 (not read by PA_ROPE_NONE), 0 < low < high and original_len >= 1 (read by
 * PA_ROPE_BANDS and PA_ROPE_RAMP only), amplitude (in fp32) and every frequency finite
 * (PA_ERR_ARG).
 */
int pa_rope_table(float* cos_sin, int64_t first_position, int64_t num_positions, int32_t rot_dim, double base,
                  int32_t scaling, double factor, int32_t original_len, double low, double high, double amplitude,
                  void* stream);

/*
 * pa_rope_and_cache - new tokens' queries and keys rotated by their
 * positions, keys and values written into their cache slots.
 *   q, k, v    : [num_tokens][heads][head_dim] of dtype, tokens q_stride,
 *                k_stride, v_stride elements apart (parts of one wider row
 *                may be given in place); 16-byte aligned, strides multiples of
 *                16 bytes (PA_ERR_ALIGN)
 *   positions  : int32 [num_tokens]
 *   slot_mapping : int64 [num_tokens], as pa_reshape_and_cache
 *   cos_sin    : float [num_positions][rot_dim], row p for position p, as
 *                pa_rope_table writes it
 *   interleaved: 0: pair i is elements i and rot_dim/2 + i of a head;
 *                otherwise elements 2 i and 2 i + 1
 *   q_out      : [num_tokens][num_q_heads][head_dim]; q itself (if q_stride is
 *                num_q_heads * head_dim), or apart from every input
 * With c, s the pair's entries, (x, y) becomes (x c - y s, y c + x s), every
 * product, sum and difference rounded to fp32, the result then to dtype;
 * elements from rot_dim on stay. A token with slot < 0 is padding: nothing of
 * it is written. A slot outside the pool records PA_ERR_BLOCK_OOB, a position
 * outside [0, num_positions) PA_ERR_SEQLEN; such a token is skipped too.
 * num_q_heads 0 caches alone (q and q_out may be NULL). rot_dim is even, 2 to
 * min(head_dim, 256); head_dim * sizeof(dtype) is a multiple of 16, head_dim
 * at most 1024, head counts at most 2^20, num_tokens * num_kv_heads at most 2^30
 * (PA_ERR_UNSUPPORTED). Two tokens with the same slot race.
 */
int pa_rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping, const float* cos_sin,
                      int32_t num_positions, int32_t rot_dim, int32_t interleaved, int64_t num_tokens, void* q_out,
                      void* k_cache, void* v_cache, int32_t num_blocks, int32_t block_size, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype, void* stream);

/* pa_rope_and_cache_fp8, pa_rope_and_cache_e5m2 - the same into 8-bit pools:
 * pa_reshape_and_cache_fp8's scale rule and its order of tokens (those of one
 * block in one run), the rotated keys encoded from fp32 (they are not rounded
 * to dtype first). head_dim 64 or 128. */
int pa_rope_and_cache_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                          const float* cos_sin, int32_t num_positions, int32_t rot_dim, int32_t interleaved,
                          int64_t num_tokens, void* q_out, void* k_cache, void* v_cache, float* kv_scales,
                          int32_t num_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, pa_dtype dtype, void* stream);
int pa_rope_and_cache_e5m2(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                           const float* cos_sin, int32_t num_positions, int32_t rot_dim, int32_t interleaved,
                           int64_t num_tokens, void* q_out, void* k_cache, void* v_cache, float* kv_scales,
                           int32_t num_blocks, int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads,
                           int32_t head_dim, pa_dtype dtype, void* stream);

/*
 * pa_block_summaries - the range of every key dimension over the tokens of a
 * block, for the blocks that hold tokens first_tokens[i] .. seq_lens[i] - 1 of
 * sequence i.
 *   first_tokens, seq_lens : int32 [num_seqs]; the summary of a block covers
 *                all its tokens below seq_lens[i], those before
 *                first_tokens[i] too; nothing is done where they are equal
 *   max_new_tokens : host upper bound of seq_lens[i] - first_tokens[i]
 *   summaries  : int8 [num_blocks][num_kv_heads][2][head_dim] (updated)
 *   summary_scales : float [num_blocks][num_kv_heads] (updated)
 * With the block's keys of one KV head: scale = max |k| / 127,
 * summaries[..][0][d] = min(ceil(max_t k[t][d] / scale), 127),
 * summaries[..][1][d] = max(floor(min_t k[t][d] / scale), -127), in fp32; codes
 * 0 where scale is 0, scale +infinity and codes 0 where a key is not finite.
 * (Over 8-bit pools a key is its code times the block's scale, in fp32.)
 * Every other entry stays as it is. Sequences that share a block give it the
 * same number of tokens. first_tokens below 0 or above seq_lens, more new
 * tokens than max_new_tokens, or a table too short record PA_ERR_SEQLEN, a
 * block outside the pool PA_ERR_BLOCK_OOB; what they name is left. fp16/bf16
 * head_dim 64 or 128, 8-bit pools 64 or 128, fp32 a multiple of 32 up to 256.
 */
int pa_block_summaries(const void* k_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                       const int32_t* first_tokens, const int32_t* seq_lens, int32_t num_seqs,
                       int32_t max_new_tokens, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                       int32_t head_dim, int8_t* summaries, float* summary_scales, pa_dtype dtype, void* stream);
int pa_block_summaries_fp8(const void* k_cache, const float* kv_scales, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* first_tokens, const int32_t* seq_lens,
                           int32_t num_seqs, int32_t max_new_tokens, int32_t num_blocks, int32_t block_size,
                           int32_t num_kv_heads, int32_t head_dim, int8_t* summaries, float* summary_scales,
                           void* stream);
int pa_block_summaries_e5m2(const void* k_cache, const float* kv_scales, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* first_tokens, const int32_t* seq_lens,
                            int32_t num_seqs, int32_t max_new_tokens, int32_t num_blocks, int32_t block_size,
                            int32_t num_kv_heads, int32_t head_dim, int8_t* summaries, float* summary_scales,
                            void* stream);

/*
 * pa_select_blocks - the blocks of every sequence and KV head that a decode
 * query attends to: its first num_sink, its last num_recent, and of the others
 * those of the highest scores, max_list_len in all.
 *   q          : [num_seqs][num_q_heads][head_dim] of dtype
 *   summaries, summary_scales : as pa_block_summaries writes them (those of the
 *                first num_sink and last num_recent blocks are not read)
 *   seq_lens   : int32 [num_seqs], 0 allowed; max_seq_len a host upper bound
 *   block_lists : int32 [num_seqs][num_kv_heads][max_list_len] (output): logical
 *                block numbers, rising, then -1
 *   list_lens  : int32 [num_seqs][num_kv_heads] (output)
 * The score of a block: every query head in 8 bits, s_q = max |q| / 127 and
 * codes = q / s_q rounded to nearest even (zeros for a head that is not all
 * finite); with I = sum_d max(code_d hi_d, code_d lo_d), a whole number, the
 * score is fl32(scale * max over the group's heads of fl32(s_q I)); 0 for a
 * block of scale 0; a block with an infinite scale comes first. Equal scores go to the lower block, so
 * results do not depend on the order in which the device runs. For attention
 * with a negative scale pass -q. A sequence of at most max_list_len blocks
 * lists them all. A sequence longer than max_seq_len or its table (or of
 * negative length) records PA_ERR_SEQLEN and lists nothing; a block outside the
 * pool records PA_ERR_BLOCK_OOB and comes last. head_dim a multiple of 32 up
 * to 256, a GQA group of at most 128, num_seqs at most 65535, num_sink +
 * num_recent at most max_list_len (PA_ERR_ARG). A sequence may have 169984
 * blocks in every shape, 378752 at head_dim 128 and up to 8 heads a group (8
 * CTAs' shared memory holds their scores; the bound is the smaller of
 * max_seq_len and the table; PA_ERR_UNSUPPORTED).
 */
int pa_select_blocks(const void* q, const int8_t* summaries, const float* summary_scales, const int32_t* block_tables,
                     int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int32_t num_blocks, int32_t max_list_len, int32_t num_sink, int32_t num_recent,
                     int32_t* block_lists, int32_t* list_lens, pa_dtype dtype, void* stream);

/*
 * pa_decode_sparse - pa_decode over listed blocks: query head h of sequence i
 * attends to the tokens below seq_lens[i] of the logical blocks
 * block_lists[i][kv head][0 .. list_lens[i][kv head] - 1].
 *   block_lists, list_lens : as pa_select_blocks writes them; any strictly
 *                rising list of a sequence's blocks will do
 *   out        : [num_seqs][num_q_heads][head_dim], apart from q; rows of an
 *                empty list are zeros
 * No workspace. An entry that is not above the one before it records
 * PA_ERR_ARG, one past the sequence's end PA_ERR_SEQLEN, a block outside the
 * pool PA_ERR_BLOCK_OOB; a list_lens outside [0, max_list_len] or a sequence
 * longer than its table PA_ERR_SEQLEN: the rows concerned are unspecified.
 * num_seqs at most 65535, max_list_len at most 2^26, a GQA group of at most
 * 128, any finite scale. fp16/bf16: head_dim 64 or 128; a softmax weight goes
 * into the second product as the sum of two numbers of the 16-bit type (within
 * 2^-15 of it for bf16, 2^-21 for fp16), over 8-bit pools with bf16 q rounded to
 * fp16 (2^-11). fp32: head_dim a multiple of 32 up to 256, exact fp32 arithmetic.
 * Results do not depend on the order in which the device runs.
 */
int pa_decode_sparse(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     int32_t max_blocks_per_seq, const int32_t* seq_lens, const int32_t* block_lists,
                     const int32_t* list_lens, int32_t max_list_len, int32_t num_seqs, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                     void* out, pa_dtype dtype, void* stream);

/* pa_decode_sparse_fp8, pa_decode_sparse_e5m2 - the same over 8-bit pools
 * (kv_scales as for pa_decode_fp8). q/out fp16 or bf16, head_dim 128. */
int pa_decode_sparse_fp8(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                         const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                         const int32_t* block_lists, const int32_t* list_lens, int32_t max_list_len,
                         int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                         int32_t block_size, int32_t num_blocks, float scale, void* out, pa_dtype dtype,
                         void* stream);
int pa_decode_sparse_e5m2(const void* q, const void* k_cache, const void* v_cache, const float* kv_scales,
                          const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                          const int32_t* block_lists, const int32_t* list_lens, int32_t max_list_len,
                          int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                          int32_t block_size, int32_t num_blocks, float scale, void* out, pa_dtype dtype,
                          void* stream);

/*
 * pa_selftest_bounded_wait — exercises the failure path every kernel relies
 * on: one warp waits on an mbarrier that nothing completes; the wait gives up
 * after limit_ns nanoseconds of device time (1 us .. 1 s, else PA_ERR_ARG),
 * records PA_ERR_TIMEOUT in the status word read by pa_get_status, and the
 * kernel returns, leaving the context usable. Nothing faults or traps.
 */
int pa_selftest_bounded_wait(int64_t limit_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
