// internal.h -- declarations shared by the host C++ and the CUDA launchers of
// libpagedkv.so.  Not part of the public ABI (include/pagedkv.h is).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>
#include <string>

#include "../../include/pagedkv.h"

namespace pkv {

// Thread-local last-error message; set_error returns the status it is given.
int set_error(int status, const std::string &msg);
int cuda_error(cudaError_t err, const char *what);
void clear_error();

// Maximum devices a pool caches descriptors for.
constexpr int kMaxDevices = 64;

// Tile height (tokens) the attention kernel stages per TMA transaction.
constexpr int kTileTokens = 16;

// pf_paged_prefill_attention without the decode kernel: at least this many
// query rows (new tokens x q-heads per kv-head) per (sequence, kv-head) take
// the tcgen05 kernel, fewer the warp-level MMA kernel.
constexpr int kTcMinRows = 128;

// Front of every attention workspace: reserved bytes; from kStateOffset on the
// count of captured launches over it (64 bits, device_common.cuh); from
// kFlagOffset on the flags of the few-rows kernel (two per warp of up to
// kFlagSms CTAs of kFlagWarps warps).  Records of every kernel lie behind it,
// so that whatever calls share a workspace -- other kernels, shapes or pool
// types -- the count stays one and a flag word holds a stamp or zero.
constexpr int kFlagSms = 256;
constexpr int kFlagWarps = 16;
constexpr size_t kStateOffset = 256;
constexpr size_t kFlagOffset = 512;
constexpr size_t kWorkspaceFront = kFlagOffset + (size_t)kFlagSms * kFlagWarps * 2 * sizeof(unsigned);

}  // namespace pkv

// Non-owning description of caller-owned K and V pools.
struct pf_pool {
    void *k_base;
    void *v_base;
    int n_layers;
    int n_blocks;
    int block_size;
    int n_kv_heads;
    int head_dim;
    int dtype;
    // PF_E4M3 pools: fp32 scales [n_layers][n_blocks][n_kv_heads], else null
    float *k_scale;
    float *v_scale;
    // TMA descriptors over K and V viewed as [rows][n_kv_heads][head_dim]
    // with rows = n_layers * n_blocks * block_size, encoded lazily per device.
    std::mutex mu;
    // per device: boxes of 1, 2, 4 kv-heads (CUDA-core consumers), then the
    // tensor-core layout for 1, 2, 4 kv-heads per item
    bool tmap_ready[pkv::kMaxDevices][6];
    CUtensorMap tmap_k[pkv::kMaxDevices][6];
    CUtensorMap tmap_v[pkv::kMaxDevices][6];
    // per device: the prompt kernels' boxes (one 64-element half of up to a
    // page of rows of one kv-head, swizzled): at most a tile of prefill_tc.cu, 16
    // rows, at most a tile of prompt_masked.cuh
    bool tmap_pf_ready[pkv::kMaxDevices][3];
    CUtensorMap tmap_pf_k[pkv::kMaxDevices][3];
    CUtensorMap tmap_pf_v[pkv::kMaxDevices][3];
};

namespace pkv {

// Device status word of the current device (a __device__ variable of this
// library); kernels OR pf_device_flag bits into it.
int *device_status_ptr();

// TMA descriptors of the pool for boxes of hg (1, 2 or 4) kv-heads, or (hg
// = 0) the tensor-core layout, on `device`, encoded on first use; *index
// receives their slot.
int encode_pool_tmaps(pf_pool *pool, int device, int hg, int *index);

struct WriteArgs {
    const pf_pool *pool;
    int layer;
    const void *k_new;
    const void *v_new;
    const int32_t *block_tables;
    int n_table_rows;
    int max_blocks;
    const int32_t *seq_idx;
    const int32_t *pos;
    int n_tokens;
};
int launch_write_kv(const WriteArgs &a, cudaStream_t stream);

// Quantising append into a PF_E4M3 pool (pf_append_kv).
struct AppendArgs {
    const pf_pool *pool;
    int layer;
    const void *k_new;
    const void *v_new;
    const int32_t *block_tables;
    int max_blocks;
    const int32_t *context_lens;
    const int32_t *cu_new;   // null: one token per sequence with a context, row s
    int n_seqs;
    int max_new;
};
int launch_append(const AppendArgs &a, cudaStream_t stream);

// Norms, rotation and cache write of a layer's new rows (pf_norm_rope_write).
// Strides in values between tokens.
struct NormRopeArgs {
    const pf_pool *pool;
    int layer;
    const void *q;           // null: no queries
    long long q_stride;
    const void *k;           // null: no keys (and no cache write)
    long long k_stride;
    const void *v;
    long long v_stride;
    int n_tokens;
    int n_q_heads;
    const float *q_weight;   // null: no norm
    const float *k_weight;
    float eps;
    const float *angles;
    int n_positions;
    int rot_dim;
    bool interleaved;
    const int32_t *rope_pos;       // null: pos
    const int32_t *block_tables;   // null: no cache write
    int n_table_rows;
    int max_blocks;
    const int32_t *seq_idx;
    const int32_t *pos;
    void *q_out;
    long long q_out_stride;
    void *k_out;             // null: K goes to the cache only
    long long k_out_stride;
};
int launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream);

// Whole-block copies: pool -> pool (both id arrays set), pool -> image
// (dst_ids null: destination i is image i of `image`), image -> pool
// (src_ids null).  Ids are device int32 arrays of n entries.
struct BlockCopyArgs {
    const pf_pool *pool;
    const int32_t *src_ids;
    const int32_t *dst_ids;
    const void *image;   // device-accessible address of the host images
    int n;
    // compaction: entries of the tables that a context uses go through
    // block_map in the same launch (null: no tables)
    const int32_t *block_map;
    int32_t *block_tables;
    int n_rows;
    int max_blocks;
    const int32_t *context_lens;
};
int launch_block_copy(const BlockCopyArgs &a, cudaStream_t stream);

// What a query sees of its context, beside what a call's `causal` says.
enum MaskKind {
    kMaskNone = 0,
    kMaskWindow = 1,   // of the tokens up to its position p: t > p - window or t < sinks
    kMaskTree = 2      // the queries are the context's last tokens, drafts: all tokens before them,
                       // and those drafts whose bits its row of the tree holds
};
struct AttnMask {
    int kind = kMaskNone;
    int window = 0;                   // 1 .. 2^30
    int sinks = 0;                    // 0 .. 2^30
    const uint64_t *tree = nullptr;   // [query token][tree_words]: bit j of word w for draft 64 w + j
    int tree_words = 0;
};

// Multi-token attention (pf_paged_prefill_attention, pf_paged_cross_attention).
struct PrefillArgs {
    const pf_pool *pool;
    int layer;
    const void *q;
    const int32_t *block_tables;
    int max_blocks;
    const int32_t *context_lens;
    const int32_t *cu_q;   // null (not causal): one query per sequence, row s
    int n_seqs;
    int max_new;
    int n_q_heads;
    float scale;
    void *out;
    int out_dtype;
    bool causal;   // the queries are the context's last tokens
    void *workspace = nullptr;   // for the parts of contexts cut over the SMs, or null: not cut
    size_t ws_bytes = 0;
    AttnMask mask = {};          // (not none: causal)
};
// Parts that the prompt kernel cuts contexts of these sizes into with a
// workspace of ws_bytes (1: none).
int prompt_splits(const pf_pool *pool, bool causal, int n_seqs, int n_q_heads, int max_blocks, int max_new, int sms,
                  size_t ws_bytes);
// Bytes of that workspace for these sizes and for smaller batches, 0 if these
// are not cut (or causal fp16).
size_t prompt_workspace_bytes(const pf_pool *pool, bool causal, int n_seqs, int n_q_heads, int max_blocks, int max_new);
int launch_prefill(const PrefillArgs &a, cudaStream_t stream);   // prefill_mma.cu (causal, fp16 pools)
int launch_prefill_tc(const PrefillArgs &a, cudaStream_t stream);   // prefill_tc.cu
// fp16 pools: the boxes of prompt kernel `which`, of box_rows rows, on first use.
int encode_prompt_tmaps(pf_pool *pool, int dev, int which, int box_rows);
// The same under a mask (prompt_masked.cu).
int masked_splits(const pf_pool *pool, const AttnMask &mask, int n_seqs, int n_q_heads, int max_blocks, int max_new,
                  int sms, size_t ws_bytes);
size_t masked_workspace_bytes(const pf_pool *pool, const AttnMask &mask, int n_seqs, int n_q_heads, int max_blocks, int max_new);
int launch_prompt_masked(const PrefillArgs &a, cudaStream_t stream);

struct GatherArgs {
    const pf_pool *pool;
    int layer;
    const int32_t *block_tables;
    int max_blocks;
    const int32_t *context_lens;
    const int64_t *cu_off;
    int n_seqs;
    void *k_out;
    void *v_out;
};
int launch_gather_kv(const GatherArgs &a, cudaStream_t stream);
int launch_gather_e4m3(const GatherArgs &a, cudaStream_t stream);

// What plain launches are stamped by, counted; whether a launch on the stream is
// captured (then stamp 0: device_common.cuh).
unsigned next_epoch();
int is_captured(cudaStream_t stream, bool *out);

// SMs of the current device; without one an error, or a bound for sizing.
int device_sms(bool need_device, int *sms);

// Attention of at most kMaxRows query rows per (sequence, kv-head):
// rows_attention.cuh.  Every schedule detail follows from the device and the
// rows; the workspace holds the parts of cut sequences.
constexpr int kMaxRows = 16;
struct RowsPlan {
    int sms;
    int grid;
    size_t bytes;   // of the workspace
};
// With as many CTAs as the device has SMs (at most kFlagSms), or fewer whose
// workspace fits into `most` bytes.
int rows_plan(const pf_pool *pool, int n_rows, bool need_device, RowsPlan *plan, size_t most = SIZE_MAX);
// pf_paged_decode_attention over an 8-bit pool on as many SMs as a scratch of
// `bytes` serves (abi.cpp).
int decode_on_scratch(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables, int max_blocks,
                      const int32_t *context_lens, int n_seqs, int n_q_heads, float scale, void *out, int out_dtype,
                      int split_tokens, void *scratch, size_t bytes, void *stream);
struct RowsArgs {
    const pf_pool *pool;
    int layer;
    const void *q;
    const int32_t *block_tables;
    int max_blocks;
    const int32_t *context_lens;
    const int32_t *cu_q;   // null: one query per sequence, row s
    int n_seqs;
    int n_q_heads;
    int rows;              // most query tokens of a sequence x q-heads per kv-head
    bool causal;           // the queries are the context's last tokens
    float scale;
    void *out;
    int out_dtype;
    RowsPlan plan;
    void *workspace;
    bool after_append;     // the stream's previous kernel is this call's append
    AttnMask mask = {};    // (not none: causal)
};
int launch_rows(const RowsArgs &a, cudaStream_t stream);

// How an attention call is scheduled and what workspace it needs.
struct AttnPlan {
    bool spans;            // balanced spans (split_tokens 0 or -2) or fixed chunks
    bool cuda_cores;       // CUDA-core consumers (split_tokens != 0): fp32 scores and weights
    int chunk;             // chunk schedule: tokens per chunk
    int grid;              // persistent grid (0 when planned without a device)
    size_t counter_bytes;  // the workspace's front (kWorkspaceFront)
    size_t partial_bytes;  // partial records (spans: 64-bit words tagged with the launch's stamp; chunks: fp32), then merge jobs
    size_t n_jobs;         // chunk schedule: merge job slots (0: no merge kernel)
};
int attention_plan(const pf_pool *pool, int n_seqs, int n_q_heads, int max_blocks, int split_tokens,
                   bool need_device, AttnPlan *plan);

struct AttnArgs {
    pf_pool *pool;
    int layer;
    const void *q;
    const void *k_new;   // fused decode step: new token rows (null: attention only)
    const void *v_new;
    bool overlap_previous;   // launch as a programmatic dependent of the previous kernel
    const int32_t *block_tables;
    int max_blocks;
    const int32_t *context_lens;
    int n_seqs;
    int n_q_heads;
    // rows per kv-head: its q-heads for decode; for an append (cu_q set),
    // the most query tokens of a sequence x its q-heads (at most 8)
    int rows;
    const int32_t *cu_q;   // append: query rows of sequence s are cu_q[s] .. cu_q[s + 1] - 1
    float scale;
    void *out;
    int out_dtype;
    AttnPlan plan;
    void *workspace;
    size_t ws_bytes;
};
int launch_attention(const AttnArgs &a, cudaStream_t stream);

}  // namespace pkv
