// abi.cpp -- C ABI entry points of libpagedkv.so that are not the allocator:
// error reporting, pool descriptors, host-side argument validation and the
// dispatch of the device calls to their launchers.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <string>

#include "internal.h"

namespace pkv {

namespace {
thread_local std::string g_last_error;
}

int set_error(int status, const std::string &msg) {
    g_last_error = msg;
    return status;
}

int cuda_error(cudaError_t err, const char *what) {
    return set_error(PF_ERR_CUDA, std::string(what) + ": " + cudaGetErrorName(err) + " (" +
                                      cudaGetErrorString(err) + ")");
}

void clear_error() { g_last_error.clear(); }

}  // namespace pkv

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_block_size(int b) { return b == 1 || b == 16 || b == 64 || b == 256; }

bool valid_head_dim(int d) { return d == 64 || d == 128; }

// Calls that exist for one pool type only.
int need_dtype(const pf_pool *pool, int dtype, const char *fn, const char *instead) {
    if (pool->dtype == dtype) return PF_OK;
    return pkv::set_error(PF_ERR_UNSUPPORTED, std::string(fn) + ": not built for " +
                                                  (pool->dtype == PF_E4M3 ? "PF_E4M3" : "PF_F16") + " pools" + instead);
}

int check_pool(const pf_pool *pool, int layer, const char *fn) {
    if (!pool) return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": pool is null");
    if (layer < 0 || layer >= pool->n_layers)
        return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": layer " + std::to_string(layer) +
                                                  " outside [0, " + std::to_string(pool->n_layers) + ")");
    return PF_OK;
}

}  // namespace

extern "C" {

const char *pf_last_error(void) { return pkv::g_last_error.c_str(); }

int pf_abi_version(void) { return PF_ABI_VERSION; }

size_t pf_pool_bytes(int n_layers, int n_blocks, int block_size, int n_kv_heads, int head_dim,
                     int dtype) {
    if (n_layers <= 0 || n_blocks <= 0 || block_size <= 0 || n_kv_heads <= 0 || head_dim <= 0 ||
        (dtype != PF_F16 && dtype != PF_E4M3))
        return 0;
    return (size_t)n_layers * (size_t)n_blocks * (size_t)block_size * (size_t)n_kv_heads *
           (size_t)head_dim * (dtype == PF_F16 ? 2u : 1u);
}

size_t pf_scale_bytes(int n_layers, int n_blocks, int n_kv_heads) {
    if (n_layers <= 0 || n_blocks <= 0 || n_kv_heads <= 0) return 0;
    return (size_t)n_layers * (size_t)n_blocks * (size_t)n_kv_heads * sizeof(float);
}

static int pool_create(pf_pool **out, void *k_base, void *v_base, float *k_scale, float *v_scale, int n_layers,
                       int n_blocks, int block_size, int n_kv_heads, int head_dim, int dtype) {
    if (!out) return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: out is null");
    *out = nullptr;
    if (!k_base || !v_base) return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: null pool pointer");
    if (!aligned16(k_base) || !aligned16(v_base))
        return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: pool pointers must be 16-byte aligned");
    if (!valid_head_dim(head_dim))
        return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: head_dim must be 64 or 128");
    if (!valid_block_size(block_size))
        return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: block_size must be 1, 16, 64 or 256");
    if (n_layers <= 0 || n_blocks <= 0 || n_kv_heads <= 0 || n_kv_heads > 256)
        return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: n_layers, n_blocks must be positive and "
                                              "n_kv_heads in [1, 256]");
    uint64_t rows = (uint64_t)n_layers * (uint64_t)n_blocks * (uint64_t)block_size;
    if (rows >= (1ull << 31))
        return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: n_layers * n_blocks * block_size must be "
                                              "below 2^31 token rows");
    pf_pool *p = new (std::nothrow) pf_pool;
    if (!p) return pkv::set_error(PF_ERR_OOM, "pf_pool_create: host allocation failed");
    p->k_base = k_base;
    p->v_base = v_base;
    p->k_scale = k_scale;
    p->v_scale = v_scale;
    p->n_layers = n_layers;
    p->n_blocks = n_blocks;
    p->block_size = block_size;
    p->n_kv_heads = n_kv_heads;
    p->head_dim = head_dim;
    p->dtype = dtype;
    for (int i = 0; i < pkv::kMaxDevices; ++i) {
        for (int j = 0; j < 6; ++j) p->tmap_ready[i][j] = false;
        p->tmap_pf_ready[i][0] = p->tmap_pf_ready[i][1] = p->tmap_pf_ready[i][2] = false;
    }
    *out = p;
    return PF_OK;
}

int pf_pool_create(pf_pool **out, void *k_base, void *v_base, int n_layers, int n_blocks, int block_size,
                   int n_kv_heads, int head_dim, int dtype) {
    pkv::clear_error();
    if (out) *out = nullptr;
    if (dtype != PF_F16)
        return pkv::set_error(PF_ERR_INVALID, "pf_pool_create: dtype must be PF_F16 (PF_E4M3 pools have scales: "
                                              "pf_pool_create_e4m3)");
    return pool_create(out, k_base, v_base, nullptr, nullptr, n_layers, n_blocks, block_size, n_kv_heads, head_dim,
                       dtype);
}

int pf_pool_create_e4m3(pf_pool **out, void *k_base, void *v_base, float *k_scale, float *v_scale, int n_layers,
                        int n_blocks, int block_size, int n_kv_heads, int head_dim) {
    pkv::clear_error();
    if (out) *out = nullptr;
    if (!k_scale || !v_scale) return pkv::set_error(PF_ERR_INVALID, "pf_pool_create_e4m3: null scale pointer");
    if (((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u) != 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_pool_create_e4m3: scale pointers must be 4-byte aligned");
    return pool_create(out, k_base, v_base, k_scale, v_scale, n_layers, n_blocks, block_size, n_kv_heads, head_dim,
                       PF_E4M3);
}

int pf_pool_destroy(pf_pool *pool) {
    pkv::clear_error();
    delete pool;
    return PF_OK;
}

int pf_write_kv(const pf_pool *pool, int layer, const void *k_new, const void *v_new,
                const int32_t *block_tables, int n_table_rows, int max_blocks_per_seq,
                const int32_t *seq_idx, const int32_t *pos, int n_tokens, void *stream) {
    pkv::clear_error();
    int rc = check_pool(pool, layer, "pf_write_kv");
    if (rc) return rc;
    if ((rc = need_dtype(pool, PF_F16, "pf_write_kv", ": pf_append_kv quantises")) != PF_OK) return rc;
    if (n_tokens < 0) return pkv::set_error(PF_ERR_INVALID, "pf_write_kv: negative n_tokens");
    if (n_tokens == 0) return PF_OK;
    if (!k_new || !v_new || !block_tables || !seq_idx || !pos)
        return pkv::set_error(PF_ERR_INVALID, "pf_write_kv: null pointer");
    if (!aligned16(k_new) || !aligned16(v_new))
        return pkv::set_error(PF_ERR_INVALID, "pf_write_kv: k_new / v_new must be 16-byte aligned");
    if (max_blocks_per_seq <= 0 || n_table_rows <= 0)
        return pkv::set_error(PF_ERR_INVALID,
                              "pf_write_kv: n_table_rows and max_blocks_per_seq must be positive");
    pkv::WriteArgs a{pool, layer, k_new, v_new, block_tables, n_table_rows, max_blocks_per_seq,
                     seq_idx, pos, n_tokens};
    return pkv::launch_write_kv(a, static_cast<cudaStream_t>(stream));
}

int pf_norm_rope_write(const pf_pool *pool, int layer, const void *q, int64_t q_stride, const void *k,
                       int64_t k_stride, const void *v, int64_t v_stride, int n_tokens, int n_q_heads,
                       const float *q_weight, const float *k_weight, float eps, const float *angles, int n_positions,
                       int rot_dim, int flags, const int32_t *rope_pos, const int32_t *block_tables, int n_table_rows,
                       int max_blocks_per_seq, const int32_t *seq_idx, const int32_t *pos, void *q_out,
                       int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream) {
    pkv::clear_error();
    const auto bad = [](const char *what) {
        return pkv::set_error(PF_ERR_INVALID, std::string("pf_norm_rope_write: ") + what);
    };
    int rc = check_pool(pool, layer, "pf_norm_rope_write");
    if (rc) return rc;
    if (flags & ~PF_ROPE_INTERLEAVED) return bad("unknown flags");
    if (n_tokens < 0) return bad("negative n_tokens");
    if (n_tokens == 0) return PF_OK;
    const int D = pool->head_dim;
    const bool cached = block_tables != nullptr;
    if (cached && (rc = need_dtype(pool, PF_F16, "pf_norm_rope_write", ": without block_tables, then pf_append_kv of k_out")) != PF_OK)
        return rc;
    if (!q && !k) return bad("neither queries nor keys");
    if (q && (n_q_heads <= 0 || !q_out)) return bad("queries need n_q_heads > 0 and q_out");
    if (q && n_q_heads > 65536) return bad("n_q_heads is too large");
    if (!q && (n_q_heads != 0 || q_out || q_weight)) return bad("n_q_heads, q_out or q_weight without q");
    if (!k && (cached || k_out || k_weight)) return bad("block_tables, k_out or k_weight without k");
    if (k && !cached && !k_out) return bad("keys need block_tables or k_out");
    if (cached && (!v || !seq_idx || !pos)) return bad("a cache write needs v, seq_idx and pos");
    if (cached && (max_blocks_per_seq <= 0 || n_table_rows <= 0))
        return bad("n_table_rows and max_blocks_per_seq must be positive");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) ||
        !aligned16(k_weight) || !aligned16(angles))
        return bad("rows, weights and angles must be 16-byte aligned");
    for (const int64_t s : {q ? q_stride : 0, k ? k_stride : 0, cached ? v_stride : 0, q ? q_out_stride : 0, k_out ? k_out_stride : 0})
        if (s < 0 || s % 8 || s > (1ll << 40)) return bad("strides must be multiples of 8 values, not negative");
    if (n_tokens > 1 && ((q && q_out_stride < (int64_t)n_q_heads * D) || (k_out && k_out_stride < (int64_t)pool->n_kv_heads * D)))
        return bad("the output rows of neighbouring tokens overlap");
    if ((q_weight || k_weight) && !(eps >= 0.0f && eps <= FLT_MAX)) return bad("eps must be a number, not negative");
    if (rot_dim < 0 || rot_dim > D) return bad("rot_dim must be in [0, head_dim]");
    if (rot_dim % 16) return pkv::set_error(PF_ERR_UNSUPPORTED, "pf_norm_rope_write: rot_dim must be a multiple of 16");
    if (rot_dim && (!angles || n_positions <= 0)) return bad("a rotation needs angles of n_positions > 0");
    if (rot_dim && !rope_pos && !pos) return bad("a rotation needs rope_pos or pos");
    pkv::NormRopeArgs a{pool, layer, q, q_stride, k, k_stride, cached ? v : nullptr, v_stride, n_tokens, n_q_heads,
                        q_weight, k_weight, eps, angles, n_positions, rot_dim, (flags & PF_ROPE_INTERLEAVED) != 0,
                        rope_pos, block_tables, n_table_rows, max_blocks_per_seq, seq_idx, pos, q_out, q_out_stride,
                        k_out, k_out_stride};
    return pkv::launch_norm_rope(a, static_cast<cudaStream_t>(stream));
}

int pf_append_kv(const pf_pool *pool, int layer, const void *k_new, const void *v_new, const int32_t *block_tables,
                 int max_blocks_per_seq, const int32_t *context_lens, const int32_t *cu_new, int n_seqs,
                 int max_new_tokens, void *stream) {
    pkv::clear_error();
    int rc = check_pool(pool, layer, "pf_append_kv");
    if (rc) return rc;
    if ((rc = need_dtype(pool, PF_E4M3, "pf_append_kv", ": pf_write_kv copies")) != PF_OK) return rc;
    if (n_seqs < 0 || max_new_tokens < 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_append_kv: negative n_seqs or max_new_tokens");
    if (n_seqs == 0 || max_new_tokens == 0) return PF_OK;
    if (!k_new || !v_new || !block_tables || !context_lens)
        return pkv::set_error(PF_ERR_INVALID, "pf_append_kv: null pointer");
    if (!aligned16(k_new) || !aligned16(v_new))
        return pkv::set_error(PF_ERR_INVALID, "pf_append_kv: k_new / v_new must be 16-byte aligned");
    if (max_blocks_per_seq <= 0 || (long long)max_blocks_per_seq * pool->block_size > (1ll << 30))
        return pkv::set_error(PF_ERR_INVALID, "pf_append_kv: bad max_blocks_per_seq");
    if (!cu_new && max_new_tokens != 1)
        return pkv::set_error(PF_ERR_INVALID, "pf_append_kv: max_new_tokens must be 1 without cu_new");
    pkv::AppendArgs a{pool, layer, k_new, v_new, block_tables, max_blocks_per_seq, context_lens, cu_new, n_seqs,
                      max_new_tokens};
    return pkv::launch_append(a, static_cast<cudaStream_t>(stream));
}

int pf_gather_kv(const pf_pool *pool, int layer, const int32_t *block_tables, int max_blocks_per_seq,
                 const int32_t *context_lens, const int64_t *cu_off, int n_seqs, void *k_out,
                 void *v_out, void *stream) {
    pkv::clear_error();
    int rc = check_pool(pool, layer, "pf_gather_kv");
    if (rc) return rc;
    if (n_seqs < 0) return pkv::set_error(PF_ERR_INVALID, "pf_gather_kv: negative n_seqs");
    if (n_seqs == 0) return PF_OK;
    if (!block_tables || !context_lens || !cu_off || !k_out || !v_out)
        return pkv::set_error(PF_ERR_INVALID, "pf_gather_kv: null pointer");
    if (!aligned16(k_out) || !aligned16(v_out))
        return pkv::set_error(PF_ERR_INVALID, "pf_gather_kv: k_out / v_out must be 16-byte aligned");
    if (max_blocks_per_seq <= 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_gather_kv: max_blocks_per_seq must be positive");
    pkv::GatherArgs a{pool, layer, block_tables, max_blocks_per_seq, context_lens, cu_off,
                      n_seqs, k_out, v_out};
    if (pool->dtype == PF_E4M3) {
        if ((long long)max_blocks_per_seq * pool->block_size > (1ll << 30))
            return pkv::set_error(PF_ERR_INVALID, "pf_gather_kv: max_blocks_per_seq is too large");
        return pkv::launch_gather_e4m3(a, static_cast<cudaStream_t>(stream));
    }
    return pkv::launch_gather_kv(a, static_cast<cudaStream_t>(stream));
}

size_t pf_block_image_bytes(const pf_pool *pool) {
    if (!pool) return 0;
    if (pool->dtype == PF_E4M3)   // codes, then the scales padded to 16 bytes
        return (size_t)pool->n_layers * 2 *
               ((size_t)pool->block_size * pool->n_kv_heads * pool->head_dim + ((size_t)pool->n_kv_heads * 4 + 15) / 16 * 16);
    return (size_t)pool->n_layers * 2 * pool->block_size * pool->n_kv_heads * pool->head_dim * sizeof(uint16_t);
}

int pf_copy_blocks(const pf_pool *pool, const int32_t *src_ids, const int32_t *dst_ids, int n, void *stream) {
    pkv::clear_error();
    if (!pool) return pkv::set_error(PF_ERR_INVALID, "pf_copy_blocks: pool is null");
    if (n < 0) return pkv::set_error(PF_ERR_INVALID, "pf_copy_blocks: negative count");
    if (n == 0) return PF_OK;
    if (!src_ids || !dst_ids) return pkv::set_error(PF_ERR_INVALID, "pf_copy_blocks: null id array");
    pkv::BlockCopyArgs a{pool, src_ids, dst_ids, nullptr, n, nullptr, nullptr, 0, 0, nullptr};
    return pkv::launch_block_copy(a, static_cast<cudaStream_t>(stream));
}

int pf_compact_blocks(const pf_pool *pool, const int32_t *src_ids, const int32_t *dst_ids, int n,
                      const int32_t *block_map, int32_t *block_tables, int n_table_rows, int max_blocks_per_seq,
                      const int32_t *context_lens, void *stream) {
    pkv::clear_error();
    if (!pool) return pkv::set_error(PF_ERR_INVALID, "pf_compact_blocks: pool is null");
    if (n < 0 || n_table_rows < 0) return pkv::set_error(PF_ERR_INVALID, "pf_compact_blocks: negative count");
    if (n > 0 && (!src_ids || !dst_ids)) return pkv::set_error(PF_ERR_INVALID, "pf_compact_blocks: null id array");
    if (n_table_rows > 0) {
        if (!block_map || !block_tables || !context_lens)
            return pkv::set_error(PF_ERR_INVALID, "pf_compact_blocks: null pointer");
        if (max_blocks_per_seq <= 0)
            return pkv::set_error(PF_ERR_INVALID, "pf_compact_blocks: max_blocks_per_seq must be positive");
    }
    if (n == 0 && n_table_rows == 0) return PF_OK;
    pkv::BlockCopyArgs a{pool,   src_ids, dst_ids, nullptr, n, block_map, n_table_rows > 0 ? block_tables : nullptr,
                         n_table_rows, max_blocks_per_seq, context_lens};
    return pkv::launch_block_copy(a, static_cast<cudaStream_t>(stream));
}

// Device address of a page-locked host buffer (its mapping), or an error.
static int host_image_ptr(const void *host, void **dev_out, const char *what) {
    if (!host) return pkv::set_error(PF_ERR_INVALID, std::string(what) + ": host buffer is null");
    if (!aligned16(host)) return pkv::set_error(PF_ERR_INVALID, std::string(what) + ": host buffer must be 16-byte aligned");
    cudaPointerAttributes attr;
    cudaError_t e = cudaPointerGetAttributes(&attr, host);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return pkv::cuda_error(e, (std::string(what) + ": cudaPointerGetAttributes").c_str());
    }
    if (attr.type != cudaMemoryTypeHost || attr.devicePointer == nullptr)
        return pkv::set_error(PF_ERR_INVALID, std::string(what) +
                                                  ": host buffer must be page-locked host memory "
                                                  "(cudaHostAlloc, cudaHostRegister or a pinned tensor)");
    *dev_out = attr.devicePointer;
    return PF_OK;
}

int pf_swap_out(const pf_pool *pool, const int32_t *ids, int n, void *host_dst, void *stream) {
    pkv::clear_error();
    if (!pool) return pkv::set_error(PF_ERR_INVALID, "pf_swap_out: pool is null");
    if (n < 0) return pkv::set_error(PF_ERR_INVALID, "pf_swap_out: negative count");
    if (n == 0) return PF_OK;
    if (!ids) return pkv::set_error(PF_ERR_INVALID, "pf_swap_out: ids is null");
    void *img = nullptr;
    int rc = host_image_ptr(host_dst, &img, "pf_swap_out");
    if (rc) return rc;
    pkv::BlockCopyArgs a{pool, ids, nullptr, img, n, nullptr, nullptr, 0, 0, nullptr};
    return pkv::launch_block_copy(a, static_cast<cudaStream_t>(stream));
}

int pf_swap_in(const pf_pool *pool, const void *host_src, const int32_t *ids, int n, void *stream) {
    pkv::clear_error();
    if (!pool) return pkv::set_error(PF_ERR_INVALID, "pf_swap_in: pool is null");
    if (n < 0) return pkv::set_error(PF_ERR_INVALID, "pf_swap_in: negative count");
    if (n == 0) return PF_OK;
    if (!ids) return pkv::set_error(PF_ERR_INVALID, "pf_swap_in: ids is null");
    void *img = nullptr;
    int rc = host_image_ptr(host_src, &img, "pf_swap_in");
    if (rc) return rc;
    pkv::BlockCopyArgs a{pool, nullptr, ids, img, n, nullptr, nullptr, 0, 0, nullptr};
    return pkv::launch_block_copy(a, static_cast<cudaStream_t>(stream));
}

// Whether rows are many enough values that the few-rows kernel pays for its
// parts more than the prompt kernel does.
static bool wide_rows(const pf_pool *pool, int rows) { return rows * pool->head_dim > 512; }

// Workspace bytes for calls of up to `rows` rows per kv-head on either kernel.
// (Fewer rows may take more: up to 8 run with 16 warps a CTA, more with 12.  The
// prompt kernel's bytes, with which it cuts as far as it likes, are those of a
// single sequence: a workspace serves smaller batches than its own.)
static size_t rows_workspace_bytes(const pf_pool *pool, int rows, int n_q_heads, int max_blocks, bool causal,
                                   const pkv::AttnMask &mask = {}) {
    const int group = n_q_heads / pool->n_kv_heads;
    size_t most = 0;
    for (int r = group; r <= rows; r += group) {
        pkv::RowsPlan plan;
        if (pkv::rows_plan(pool, r, false, &plan) != PF_OK) return 0;
        most = std::max(most, plan.bytes);
        if (wide_rows(pool, r))
            most = std::max(most, mask.kind == pkv::kMaskNone
                                      ? pkv::prompt_workspace_bytes(pool, causal, 1, n_q_heads, max_blocks, r / group)
                                      : pkv::masked_workspace_bytes(pool, mask, 1, n_q_heads, max_blocks, r / group));
    }
    return most;
}

// The same for calls on the prompt kernel alone: 0, or enough for calls of
// fewer rows too.
static size_t prompt_or_rows_workspace_bytes(const pf_pool *pool, bool causal, int n_seqs, int n_q_heads,
                                             int max_blocks, int max_tokens, const pkv::AttnMask &mask = {}) {
    const size_t bytes = mask.kind == pkv::kMaskNone
                             ? pkv::prompt_workspace_bytes(pool, causal, n_seqs, n_q_heads, max_blocks, max_tokens)
                             : pkv::masked_workspace_bytes(pool, mask, n_seqs, n_q_heads, max_blocks, max_tokens);
    return bytes == 0 ? 0 : std::max(bytes, rows_workspace_bytes(pool, pkv::kMaxRows, n_q_heads, max_blocks, causal, mask));
}

size_t pf_decode_workspace_bytes(const pf_pool *pool, int n_seqs, int n_q_heads, int max_blocks_per_seq,
                                 int split_tokens) {
    pkv::clear_error();
    if (!pool || n_seqs <= 0 || n_q_heads <= 0 || max_blocks_per_seq <= 0 ||
        n_q_heads % pool->n_kv_heads) {
        pkv::set_error(PF_ERR_INVALID, "pf_decode_workspace_bytes: bad arguments");
        return 0;
    }
    if (pool->dtype == PF_E4M3) {
        const int group = n_q_heads / pool->n_kv_heads;
        if (group > pkv::kMaxRows || split_tokens != 0) {
            pkv::set_error(PF_ERR_UNSUPPORTED, "pf_decode_workspace_bytes: PF_E4M3 pools take split_tokens = 0 and "
                                               "at most 16 q-heads per kv-head");
            return 0;
        }
        return rows_workspace_bytes(pool, group, n_q_heads, max_blocks_per_seq, false);
    }
    pkv::AttnPlan plan;
    if (pkv::attention_plan(pool, n_seqs, n_q_heads, max_blocks_per_seq, split_tokens, false, &plan)) return 0;
    return plan.counter_bytes + plan.partial_bytes;
}

int pf_decode_workspace_init(void *workspace, size_t ws_bytes, void *stream) {
    pkv::clear_error();
    if (!workspace || ws_bytes == 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_decode_workspace_init: null or empty workspace");
    cudaError_t e = cudaMemsetAsync(workspace, 0, ws_bytes, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv::cuda_error(e, "pf_decode_workspace_init: cudaMemsetAsync");
    return PF_OK;
}

// Whether a call of few rows takes the prompt kernel, whose blocks (one per
// sequence and kv-head) need no partition and no merge, instead of a cut over
// all SMs.  A wave of its blocks takes about 4 + steps microseconds, steps of
// 128 tokens (64 at head_dim 128; twice as many where fp16 pages hold one
// token each) at the table's longest context.  Measured, 8 kv-heads, few-rows
// kernel / prompt kernel in microseconds:
//   4 sequences, 1 row x 64 values, fp16: 100 tokens 10.9 / 5.8, 1024 tokens
//   14.4 / 12.3, 1536 tokens 14.9 / 15.9; x 128, e4m3: 512 tokens 14.7 / 12.1,
//   1024 tokens 17.0 / 19.2; 16 rows x 128, fp16: 512 tokens 31.8 / 11.1, 2048
//   tokens 47.7 / 30.8 (cut into parts 16.2), 8192 tokens 59.6 / 109 (36.5); 9
//   rows x 64: 2048 tokens 23.2 / 19.6 (13.7);
//   38 sequences (two waves), 1 row x 64, e4m3: 128 tokens 10.4 / 12.5; 16 rows
//   x 128, fp16: 256 tokens 27.7 / 16.4, 1024 tokens, e4m3 38.6 / 39.1; 32
//   sequences of 512 tokens, e4m3 x 128: 8 rows 22.5 / 23.8, 9 25.9 / 23.9;
//   38 of 512 tokens, e4m3 x 64: 9 rows 18.2 / 19.0, 16 19.5 / 19.2.
// So at its border the rule is a few per cent from the better kernel either way
// (two waves of 9 rows x 64 and 512 tokens take the prompt kernel, 4 % slower).
// The table's width stands for the contexts, which the host does not know: over
// tables much wider than their contexts few rows stay with the few-rows kernel.
// fp32 results stay with the few-rows kernel, which does not round its weights
// to fp16.
static bool prompt_kernel_pays(const pkv::RowsArgs &a, size_t ws_bytes) {
    if (a.out_dtype != PF_F16) return false;
    const long long items = (long long)a.n_seqs * a.pool->n_kv_heads;
    const long long waves = (items + a.plan.sms - 1) / a.plan.sms;
    const int step = a.pool->head_dim == 64 ? 128 : 64;
    long long steps = ((long long)a.max_blocks * a.pool->block_size + step - 1) / step;
    if (a.pool->block_size < 16 && a.pool->dtype == PF_F16) steps *= 2;
    if (!wide_rows(a.pool, a.rows)) return waves == 1 && steps <= 8;
    if (waves > 1) return waves == 2 && steps <= (a.rows * a.pool->head_dim > 1024 ? 8 : 4);
    return steps <= 32 || pkv::prompt_splits(a.pool, a.causal && a.cu_q, a.n_seqs, a.n_q_heads, a.max_blocks,
                                             a.rows / (a.n_q_heads / a.pool->n_kv_heads), a.plan.sms, ws_bytes) > 1;
}

// The same for calls under a mask, whose prompt kernel stays on the SMs: its later
// waves cost less.  Both kernels' microseconds at the longest contexts (a
// window's tokens), fitted to 8 kv-heads, 1 to 16 rows, 4 to 64 sequences, 128 to
// 2,112 tokens seen, both head_dims and types, pages of 1 and 16 (272 cases): the
// choice costs 0.4 % on average and 28 % at most.  Few-rows kernel / prompt kernel: 16 sequences, window
// 2,048, 16 rows x 128 fp16 52.4 / 29.1, 1 row 32.0 / 28.9, x 64 17.8 / 18.5; 64
// sequences, window 512, 16 rows x 128 45.3 / 37.8, 7 rows 34.6 / 37.7, 1 row x 64 16.1 /
// 29.5; 32 trees of 16 drafts, 1,024 tokens, x 128 e4m3 39.7 / 30.0, x 64 23.4 / 25.1.
static bool masked_prompt_pays(const pkv::RowsArgs &a, size_t ws_bytes) {
    if (a.out_dtype != PF_F16) return false;
    const int D = a.pool->head_dim;
    const bool q8 = a.pool->dtype == PF_E4M3;
    const long long items = (long long)a.n_seqs * a.pool->n_kv_heads;
    const long long waves = (items + a.plan.sms - 1) / a.plan.sms;
    const int tile = D == 64 ? 128 : 64;
    long long tiles = ((long long)a.max_blocks * a.pool->block_size + tile - 1) / tile;
    if (a.mask.kind == pkv::kMaskWindow)   // a block's: its sinks, and its window (and one of either is cut)
        tiles = std::min(tiles, (a.mask.sinks + tile - 1ll) / tile + (a.mask.window + tile - 1ll) / tile + 1);
    const double tokens = (double)(tiles * tile), bytes = (double)items * tokens * D * (q8 ? 2 : 4);
    if (a.pool->block_size < 16 && !q8) tiles *= 2;
    const int parts = pkv::masked_splits(a.pool, a.mask, a.n_seqs, a.n_q_heads, a.max_blocks,
                                         a.rows / (a.n_q_heads / a.pool->n_kv_heads), a.plan.sms, ws_bytes);
    const double per_tile = q8 ? (D == 64 ? 1.15 : 0.8) : (D == 64 ? 0.75 : 0.67);
    const double prompt = parts > 1 ? 10.5 + per_tile * (double)((tiles + parts - 1) / parts)
                                    : 4.5 + (double)waves * (2.3 + per_tile * (double)tiles);
    const double doublings = std::max(0.0, std::log2(tokens / 160.0));
    const double more_rows = std::max(0, a.rows * D - 300) * 1e-3 * (7.0 + 0.6 * doublings * doublings);
    const double few = std::max(10.0 + std::min(5.0, 2.0 * doublings) + more_rows, 10.0 + bytes / 7e6 + 0.65 * more_rows);
    return prompt < few;
}

// The few-rows kernel with a checked workspace (decode and short appends over
// PF_E4M3 pools, short cross attention), or for small calls the prompt kernel.
static int rows_call(pkv::RowsArgs &a, void *workspace, size_t ws_bytes, const char *fn, void *stream,
                     bool fit = false) {
    if (!aligned16(workspace))
        return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": workspace must be 16-byte aligned");
    if (a.max_blocks <= 0 || (long long)a.max_blocks * a.pool->block_size > (1ll << 30))
        return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": bad max_blocks_per_seq");
    int rc = pkv::rows_plan(a.pool, a.rows, true, &a.plan, fit ? ws_bytes : SIZE_MAX);
    if (rc) return rc;
    if (ws_bytes < a.plan.bytes)
        return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": workspace has " + std::to_string(ws_bytes) +
                                                  " bytes, needs " + std::to_string(a.plan.bytes));
    if (a.mask.kind == pkv::kMaskNone ? prompt_kernel_pays(a, ws_bytes) : masked_prompt_pays(a, ws_bytes)) {
        pkv::PrefillArgs b{a.pool, a.layer, a.q, a.block_tables, a.max_blocks, a.context_lens, a.cu_q, a.n_seqs,
                           a.rows / (a.n_q_heads / a.pool->n_kv_heads), a.n_q_heads, a.scale, a.out, a.out_dtype,
                           a.causal && a.cu_q, workspace, ws_bytes, a.mask};
        return a.mask.kind == pkv::kMaskNone ? pkv::launch_prefill_tc(b, static_cast<cudaStream_t>(stream))
                                             : pkv::launch_prompt_masked(b, static_cast<cudaStream_t>(stream));
    }
    a.workspace = workspace;
    return pkv::launch_rows(a, static_cast<cudaStream_t>(stream));
}

// Checks and launch shared by pf_paged_decode_attention (k_new = v_new =
// null) and pf_decode_step (the fused write of the new token rows).
static int decode_call(const pf_pool *pool, int layer, const void *q, const void *k_new, const void *v_new,
                       bool overlap_previous, const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                       int n_seqs, int n_q_heads, float scale, void *out, int out_dtype, int split_tokens,
                       void *workspace, size_t ws_bytes, void *stream, bool fit = false) {
    int rc = check_pool(pool, layer, "pf_paged_decode_attention");
    if (rc) return rc;
    if (n_seqs < 0) return pkv::set_error(PF_ERR_INVALID, "pf_paged_decode_attention: negative n_seqs");
    if (n_seqs == 0) return PF_OK;
    if (!q || !block_tables || !context_lens || !out || !workspace)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_decode_attention: null pointer");
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
        return pkv::set_error(PF_ERR_INVALID,
                              "pf_paged_decode_attention: q, out and workspace must be 16-byte aligned");
    if (out_dtype != PF_F16 && out_dtype != PF_F32)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_decode_attention: out_dtype must be PF_F16 or PF_F32");
    if (n_q_heads <= 0 || n_q_heads % pool->n_kv_heads)
        return pkv::set_error(PF_ERR_INVALID,
                              "pf_paged_decode_attention: n_q_heads must be a positive multiple of n_kv_heads");
    int group = n_q_heads / pool->n_kv_heads;
    if (group > 16 || (group > 8 && (split_tokens != 0 || (pool->block_size < 16 && pool->dtype == PF_F16))))
        return pkv::set_error(PF_ERR_UNSUPPORTED,
                              "pf_paged_decode_attention: at most 8 q-heads per kv-head are built (16 with "
                              "split_tokens = 0 and pages of at least 16 tokens)");
    if (max_blocks_per_seq <= 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_decode_attention: max_blocks_per_seq must be positive");
    if (!(scale > 0.0f) || scale != scale)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_decode_attention: scale must be a positive number");
    if (pool->dtype == PF_E4M3) {
        if (split_tokens != 0)
            return pkv::set_error(PF_ERR_UNSUPPORTED,
                                  "pf_paged_decode_attention: PF_E4M3 pools take split_tokens = 0");
        pkv::RowsArgs a{pool, layer, q, block_tables, max_blocks_per_seq, context_lens, nullptr, n_seqs, n_q_heads,
                        group, true, scale, out, out_dtype, {}, nullptr, false};
        if (k_new) {
            // the append first: a launch of its own, since a page's new scale is needed before any of its rows
            pkv::AppendArgs w{pool, layer, k_new, v_new, block_tables, max_blocks_per_seq, context_lens, nullptr,
                              n_seqs, 1};
            if ((rc = pkv::rows_plan(pool, group, true, &a.plan)) != PF_OK) return rc;
            if (ws_bytes < a.plan.bytes)   // nothing is launched by a call that fails
                return pkv::set_error(PF_ERR_INVALID, "pf_decode_step: workspace has " + std::to_string(ws_bytes) +
                                                          " bytes, needs " + std::to_string(a.plan.bytes));
            if ((long long)max_blocks_per_seq * pool->block_size > (1ll << 30))
                return pkv::set_error(PF_ERR_INVALID, "pf_decode_step: bad max_blocks_per_seq");
            rc = pkv::launch_append(w, static_cast<cudaStream_t>(stream));
            if (rc) return rc;
            a.after_append = true;
        }
        return rows_call(a, workspace, ws_bytes, "pf_paged_decode_attention", stream, fit);
    }
    pkv::AttnPlan plan;
    // host-only checks first (no device query), then the device-sized plan
    rc = pkv::attention_plan(pool, n_seqs, n_q_heads, max_blocks_per_seq, split_tokens, false, &plan);
    if (rc) return rc;
    if (ws_bytes < plan.counter_bytes)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_decode_attention: workspace has " +
                                                  std::to_string(ws_bytes) + " bytes, needs at least " +
                                                  std::to_string(plan.counter_bytes));
    rc = pkv::attention_plan(pool, n_seqs, n_q_heads, max_blocks_per_seq, split_tokens, true, &plan);
    if (rc) return rc;
    const size_t need = plan.counter_bytes + plan.partial_bytes;
    if (ws_bytes < need)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_decode_attention: workspace has " +
                                                  std::to_string(ws_bytes) + " bytes, needs " +
                                                  std::to_string(need));
    pkv::AttnArgs a{const_cast<pf_pool *>(pool), layer, q, k_new, v_new, overlap_previous, block_tables,
                    max_blocks_per_seq, context_lens, n_seqs, n_q_heads, n_q_heads / pool->n_kv_heads, nullptr,
                    scale, out, out_dtype, plan, workspace, ws_bytes};
    return pkv::launch_attention(a, static_cast<cudaStream_t>(stream));
}

int pf_paged_decode_attention(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables,
                              int max_blocks_per_seq, const int32_t *context_lens, int n_seqs, int n_q_heads,
                              float scale, void *out, int out_dtype, int split_tokens, void *workspace,
                              size_t ws_bytes, void *stream) {
    pkv::clear_error();
    return decode_call(pool, layer, q, nullptr, nullptr, false, block_tables, max_blocks_per_seq, context_lens, n_seqs,
                       n_q_heads, scale, out, out_dtype, split_tokens, workspace, ws_bytes, stream);
}

int pf_decode_step(const pf_pool *pool, int layer, const void *q, const void *k_new, const void *v_new,
                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens, int n_seqs,
                   int n_q_heads, float scale, void *out, int out_dtype, int split_tokens, void *workspace,
                   size_t ws_bytes, int flags, void *stream) {
    pkv::clear_error();
    if (flags & ~PF_STEP_OVERLAP_PREVIOUS)
        return pkv::set_error(PF_ERR_INVALID, "pf_decode_step: unknown flags " + std::to_string(flags));
    if (n_seqs > 0) {
        if (!k_new || !v_new) return pkv::set_error(PF_ERR_INVALID, "pf_decode_step: null k_new / v_new");
        if (!aligned16(k_new) || !aligned16(v_new))
            return pkv::set_error(PF_ERR_INVALID, "pf_decode_step: k_new / v_new must be 16-byte aligned");
    }
    // the same checks as pf_paged_decode_attention, then the fused launch
    return decode_call(pool, layer, q, k_new, v_new, (flags & PF_STEP_OVERLAP_PREVIOUS) != 0, block_tables,
                       max_blocks_per_seq, context_lens, n_seqs,
                       n_q_heads, scale, out, out_dtype, split_tokens, workspace, ws_bytes, stream);
}

// Query rows of a (sequence, kv-head) that a call allows, counted in 32 bits by
// the kernels: refused above (a whole block of rows more has to fit).
static int check_query_rows(const pf_pool *pool, int max_tokens, int n_q_heads, const char *fn) {
    if ((long long)max_tokens * (n_q_heads / pool->n_kv_heads) <= INT_MAX - 512) return PF_OK;
    return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": too many query tokens x q-heads per kv-head");
}

// Hands the prompt kernel a workspace to cut contexts with, as many parts as fit.
static int prompt_workspace(pkv::PrefillArgs &a, void *workspace, size_t ws_bytes, const char *fn) {
    // (causal fp16 contexts are not cut, but under a mask)
    if (!workspace || (a.causal && a.mask.kind == pkv::kMaskNone && a.pool->dtype == PF_F16)) return PF_OK;
    if (!aligned16(workspace))
        return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": workspace must be 16-byte aligned");
    a.workspace = workspace;
    a.ws_bytes = ws_bytes;
    return PF_OK;
}

// Rows per kv-head when an append takes the decode kernel (its query tokens
// x its q-heads), or 0 when they do not fit (the standalone kernel then).
// Rows per kv-head of an append on the decode kernel (query tokens x
// q-heads): up to 16 on pages of at least 16 tokens (the tensor-core
// consumers take 9 and more), up to 8 otherwise; 0 = too many.
static int append_rows(const pf_pool *pool, int n_q_heads, int max_new_tokens) {
    if (n_q_heads <= 0 || n_q_heads % pool->n_kv_heads) return 0;
    const long long rows = (long long)max_new_tokens * (n_q_heads / pool->n_kv_heads);
    const int cap = pool->block_size >= 16 || pool->dtype == PF_E4M3 ? 16 : 8;
    return rows >= 1 && rows <= cap ? (int)rows : 0;
}

size_t pf_prefill_workspace_bytes(const pf_pool *pool, int n_seqs, int n_q_heads, int max_blocks_per_seq,
                                  int max_new_tokens) {
    pkv::clear_error();
    if (!pool || n_seqs < 0 || max_blocks_per_seq <= 0 || max_new_tokens < 0) {
        pkv::set_error(PF_ERR_INVALID, "pf_prefill_workspace_bytes: bad arguments");
        return 0;
    }
    const int rows = append_rows(pool, n_q_heads, max_new_tokens);
    if (rows == 0)   // the prompt kernel, which needs none but for long contexts cut over the SMs
        return prompt_or_rows_workspace_bytes(pool, true, n_seqs, n_q_heads, max_blocks_per_seq, max_new_tokens);
    if (pool->dtype == PF_E4M3) {
        return rows_workspace_bytes(pool, rows, n_q_heads, max_blocks_per_seq, true);
    }
    // sized like pf_decode_workspace_bytes, by the resident grid, or by a bound
    // on it when no device can be queried; the most that any count of tokens up
    // to this one takes (above 8 rows of 128 values the kernel serves fewer heads
    // at a time, whose records are smaller)
    const int group = n_q_heads / pool->n_kv_heads;
    size_t most = 0;
    for (int r = group; r <= rows; r += group) {
        pkv::AttnPlan plan;
        if (pkv::attention_plan(pool, n_seqs, r * pool->n_kv_heads, max_blocks_per_seq, 0, false, &plan) != PF_OK)
            return 0;
        most = std::max(most, plan.counter_bytes + plan.partial_bytes);
    }
    return most;
}

int pf_paged_prefill_attention(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *context_lens, const int32_t *cu_q, int n_seqs,
                               int max_new_tokens, int n_q_heads, float scale, void *out, int out_dtype,
                               void *workspace, size_t ws_bytes, void *stream) {
    pkv::clear_error();
    int rc = check_pool(pool, layer, "pf_paged_prefill_attention");
    if (rc) return rc;
    if (n_seqs < 0 || max_new_tokens < 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: negative n_seqs or max_new_tokens");
    if (n_seqs == 0 || max_new_tokens == 0) return PF_OK;
    if (!q || !block_tables || !context_lens || !cu_q || !out)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: null pointer");
    if (!aligned16(q) || !aligned16(out))
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: q and out must be 16-byte aligned");
    if (out_dtype != PF_F16 && out_dtype != PF_F32)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: out_dtype must be PF_F16 or PF_F32");
    if (n_q_heads <= 0 || n_q_heads % pool->n_kv_heads)
        return pkv::set_error(PF_ERR_INVALID,
                              "pf_paged_prefill_attention: n_q_heads must be a positive multiple of n_kv_heads");
    if (n_q_heads / pool->n_kv_heads > 16)
        return pkv::set_error(PF_ERR_UNSUPPORTED, "pf_paged_prefill_attention: at most 16 q-heads per kv-head are built");
    if (max_blocks_per_seq <= 0 || (long long)max_blocks_per_seq * pool->block_size > (1ll << 30))
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: bad max_blocks_per_seq");
    if (!(scale > 0.0f) || scale != scale)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: scale must be a positive number");
    const int rows = append_rows(pool, n_q_heads, max_new_tokens);
    if (workspace != nullptr && rows > 0 && pool->dtype == PF_E4M3) {
        pkv::RowsArgs a{pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, n_q_heads,
                        rows, true, scale, out, out_dtype, {}, nullptr, false};
        return rows_call(a, workspace, ws_bytes, "pf_paged_prefill_attention", stream);
    }
    if (workspace != nullptr && rows > 0) {
        // The decode kernel, its G rows per kv-head being the query tokens x
        // q-heads: balanced spans over the contexts, merged in the kernel.
        if (!aligned16(workspace))
            return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: workspace must be 16-byte aligned");
        pkv::AttnPlan plan;
        rc = pkv::attention_plan(pool, n_seqs, rows * pool->n_kv_heads, max_blocks_per_seq, 0, true, &plan);
        if (rc) return rc;
        const size_t need = plan.counter_bytes + plan.partial_bytes;
        if (ws_bytes < need)
            return pkv::set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: workspace has " +
                                                      std::to_string(ws_bytes) + " bytes, needs " +
                                                      std::to_string(need));
        pkv::AttnArgs a{const_cast<pf_pool *>(pool), layer, q, nullptr, nullptr, false, block_tables,
                        max_blocks_per_seq, context_lens, n_seqs, n_q_heads, rows, cu_q, scale, out, out_dtype, plan,
                        workspace, ws_bytes};
        return pkv::launch_attention(a, static_cast<cudaStream_t>(stream));
    }
    // a loose bound: there are no more new tokens than the table holds
    if (check_query_rows(pool, max_new_tokens, n_q_heads, "pf_paged_prefill_attention") != PF_OK) {
        max_new_tokens = std::min(max_new_tokens, max_blocks_per_seq * pool->block_size);
        if ((rc = check_query_rows(pool, max_new_tokens, n_q_heads, "pf_paged_prefill_attention")) != PF_OK) return rc;
        pkv::clear_error();
    }
    pkv::PrefillArgs a{pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, max_new_tokens,
                       n_q_heads, scale, out, out_dtype, true};
    if ((rc = prompt_workspace(a, workspace, ws_bytes, "pf_paged_prefill_attention")) != PF_OK) return rc;
    return pkv::launch_prefill(a, static_cast<cudaStream_t>(stream));
}

// Rows per kv-head of cross attention on the few-rows kernel, 0 = too many.
static int cross_rows(const pf_pool *pool, int n_q_heads, int max_q_tokens) {
    if (n_q_heads <= 0 || n_q_heads % pool->n_kv_heads) return 0;
    const long long rows = (long long)max_q_tokens * (n_q_heads / pool->n_kv_heads);
    return rows >= 1 && rows <= pkv::kMaxRows ? (int)rows : 0;
}

size_t pf_cross_workspace_bytes(const pf_pool *pool, int n_seqs, int n_q_heads, int max_blocks_per_seq,
                                int max_q_tokens) {
    pkv::clear_error();
    if (!pool || n_seqs < 0 || max_blocks_per_seq <= 0 || max_q_tokens < 0) {
        pkv::set_error(PF_ERR_INVALID, "pf_cross_workspace_bytes: bad arguments");
        return 0;
    }
    const int rows = cross_rows(pool, n_q_heads, max_q_tokens);
    if (rows == 0)   // the prompt kernel, which needs none but for long contexts cut over the SMs
        return prompt_or_rows_workspace_bytes(pool, false, n_seqs, n_q_heads, max_blocks_per_seq, max_q_tokens);
    return rows_workspace_bytes(pool, rows, n_q_heads, max_blocks_per_seq, false);
}

int pf_paged_cross_attention(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables,
                             int max_blocks_per_seq, const int32_t *context_lens, const int32_t *cu_q, int n_seqs,
                             int max_q_tokens, int n_q_heads, float scale, void *out, int out_dtype, void *workspace,
                             size_t ws_bytes, void *stream) {
    pkv::clear_error();
    int rc = check_pool(pool, layer, "pf_paged_cross_attention");
    if (rc) return rc;
    if (n_seqs < 0 || max_q_tokens < 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_cross_attention: negative n_seqs or max_q_tokens");
    if (n_seqs == 0 || max_q_tokens == 0) return PF_OK;
    if (!q || !block_tables || !context_lens || !cu_q || !out)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_cross_attention: null pointer");
    if (!aligned16(q) || !aligned16(out))
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_cross_attention: q and out must be 16-byte aligned");
    if (out_dtype != PF_F16 && out_dtype != PF_F32)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_cross_attention: out_dtype must be PF_F16 or PF_F32");
    if (n_q_heads <= 0 || n_q_heads % pool->n_kv_heads)
        return pkv::set_error(PF_ERR_INVALID,
                              "pf_paged_cross_attention: n_q_heads must be a positive multiple of n_kv_heads");
    if (n_q_heads / pool->n_kv_heads > pkv::kMaxRows)
        return pkv::set_error(PF_ERR_UNSUPPORTED, "pf_paged_cross_attention: at most 16 q-heads per kv-head are built");
    if (max_blocks_per_seq <= 0 || (long long)max_blocks_per_seq * pool->block_size > (1ll << 30))
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_cross_attention: bad max_blocks_per_seq");
    if (!(scale > 0.0f))
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_cross_attention: scale must be a positive number");
    if ((rc = check_query_rows(pool, max_q_tokens, n_q_heads, "pf_paged_cross_attention")) != PF_OK) return rc;
    const int rows = cross_rows(pool, n_q_heads, max_q_tokens);
    if (workspace != nullptr && rows > 0) {
        pkv::RowsArgs a{pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, n_q_heads,
                        rows, false, scale, out, out_dtype, {}, nullptr, false};
        return rows_call(a, workspace, ws_bytes, "pf_paged_cross_attention", stream);
    }
    pkv::PrefillArgs a{pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, max_q_tokens,
                       n_q_heads, scale, out, out_dtype, false};
    if ((rc = prompt_workspace(a, workspace, ws_bytes, "pf_paged_cross_attention")) != PF_OK) return rc;
    return pkv::launch_prefill(a, static_cast<cudaStream_t>(stream));
}

// Checks and launch that masked attention calls share; max_tokens bounds the
// query tokens of a sequence.
static int masked_call(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables,
                       int max_blocks_per_seq, const int32_t *context_lens, const int32_t *cu_q, int n_seqs,
                       int max_tokens, int n_q_heads, float scale, const pkv::AttnMask &mask, void *out, int out_dtype,
                       void *workspace, size_t ws_bytes, const char *fn, void *stream) {
    const auto bad = [fn](const char *what) { return pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": " + what); };
    if (!q || !block_tables || !context_lens || !out) return bad("null pointer");
    if (!aligned16(q) || !aligned16(out)) return bad("q and out must be 16-byte aligned");
    if (out_dtype != PF_F16 && out_dtype != PF_F32) return bad("out_dtype must be PF_F16 or PF_F32");
    if (n_q_heads <= 0 || n_q_heads % pool->n_kv_heads) return bad("n_q_heads must be a positive multiple of n_kv_heads");
    if (n_q_heads / pool->n_kv_heads > pkv::kMaxRows)
        return pkv::set_error(PF_ERR_UNSUPPORTED, std::string(fn) + ": at most 16 q-heads per kv-head are built");
    if (max_blocks_per_seq <= 0 || (long long)max_blocks_per_seq * pool->block_size > (1ll << 30))
        return bad("bad max_blocks_per_seq");
    if (!(scale > 0.0f)) return bad("scale must be a positive number");
    // a loose bound: there are no more query tokens than the table holds
    max_tokens = std::min(max_tokens, max_blocks_per_seq * pool->block_size);
    int rc = check_query_rows(pool, max_tokens, n_q_heads, fn);
    if (rc) return rc;
    const int rows = cross_rows(pool, n_q_heads, max_tokens);
    if (workspace != nullptr && rows > 0) {
        pkv::RowsArgs a{pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, n_q_heads,
                        rows, true, scale, out, out_dtype, {}, nullptr, false, mask};
        return rows_call(a, workspace, ws_bytes, fn, stream);
    }
    pkv::PrefillArgs a{pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, max_tokens,
                       n_q_heads, scale, out, out_dtype, true, nullptr, 0, mask};
    if ((rc = prompt_workspace(a, workspace, ws_bytes, fn)) != PF_OK) return rc;
    return pkv::launch_prompt_masked(a, static_cast<cudaStream_t>(stream));
}

// Their workspaces' bytes.
static size_t masked_call_workspace_bytes(const pf_pool *pool, int n_seqs, int n_q_heads, int max_blocks_per_seq,
                                     int max_tokens, const pkv::AttnMask &mask, const char *fn) {
    if (!pool || n_seqs < 0 || max_blocks_per_seq <= 0 || max_tokens < 0) {
        pkv::set_error(PF_ERR_INVALID, std::string(fn) + ": bad arguments");
        return 0;
    }
    max_tokens = (int)std::min<long long>(max_tokens, (long long)max_blocks_per_seq * pool->block_size);
    const int rows = cross_rows(pool, n_q_heads, max_tokens);
    if (rows == 0)   // the prompt kernel, which needs none but for long contexts cut over the SMs
        return prompt_or_rows_workspace_bytes(pool, true, n_seqs, n_q_heads, max_blocks_per_seq, max_tokens, mask);
    return rows_workspace_bytes(pool, rows, n_q_heads, max_blocks_per_seq, true, mask);
}

static bool window_mask(int window, int n_sinks, pkv::AttnMask *mask) {
    if (window < 1 || n_sinks < 0) return false;
    mask->kind = pkv::kMaskWindow;
    mask->window = std::min(window, 1 << 30);   // no context is longer
    mask->sinks = std::min(n_sinks, 1 << 30);
    return true;
}

size_t pf_window_workspace_bytes(const pf_pool *pool, int n_seqs, int n_q_heads, int max_blocks_per_seq,
                                 int max_new_tokens, int window, int n_sinks) {
    pkv::clear_error();
    pkv::AttnMask mask;
    if (!window_mask(window, n_sinks, &mask)) {
        pkv::set_error(PF_ERR_INVALID, "pf_window_workspace_bytes: window must be positive, n_sinks not negative");
        return 0;
    }
    return masked_call_workspace_bytes(pool, n_seqs, n_q_heads, max_blocks_per_seq, max_new_tokens, mask,
                                  "pf_window_workspace_bytes");
}

int pf_paged_window_attention(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables,
                              int max_blocks_per_seq, const int32_t *context_lens, const int32_t *cu_q, int n_seqs,
                              int max_new_tokens, int n_q_heads, float scale, int window, int n_sinks, void *out,
                              int out_dtype, void *workspace, size_t ws_bytes, void *stream) {
    pkv::clear_error();
    const char *fn = "pf_paged_window_attention";
    int rc = check_pool(pool, layer, fn);
    if (rc) return rc;
    if (n_seqs < 0 || max_new_tokens < 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_window_attention: negative n_seqs or max_new_tokens");
    pkv::AttnMask mask;
    if (!window_mask(window, n_sinks, &mask))
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_window_attention: window must be positive, n_sinks not negative");
    if (n_seqs == 0 || max_new_tokens == 0) return PF_OK;
    if (!cu_q && max_new_tokens != 1)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_window_attention: max_new_tokens must be 1 without cu_q");
    return masked_call(pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, max_new_tokens,
                       n_q_heads, scale, mask, out, out_dtype, workspace, ws_bytes, fn, stream);
}

size_t pf_tree_workspace_bytes(const pf_pool *pool, int n_seqs, int n_q_heads, int max_blocks_per_seq,
                               int max_draft_tokens) {
    pkv::clear_error();
    pkv::AttnMask mask;
    mask.kind = pkv::kMaskTree;
    return masked_call_workspace_bytes(pool, n_seqs, n_q_heads, max_blocks_per_seq, max_draft_tokens, mask,
                                  "pf_tree_workspace_bytes");
}

int pf_paged_tree_attention(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables,
                            int max_blocks_per_seq, const int32_t *context_lens, const int32_t *cu_q, int n_seqs,
                            int max_draft_tokens, int n_q_heads, float scale, const uint64_t *tree, int tree_words,
                            void *out, int out_dtype, void *workspace, size_t ws_bytes, void *stream) {
    pkv::clear_error();
    const char *fn = "pf_paged_tree_attention";
    int rc = check_pool(pool, layer, fn);
    if (rc) return rc;
    if (n_seqs < 0 || max_draft_tokens < 0)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_tree_attention: negative n_seqs or max_draft_tokens");
    if (n_seqs == 0 || max_draft_tokens == 0) return PF_OK;
    if (!cu_q || !tree) return pkv::set_error(PF_ERR_INVALID, "pf_paged_tree_attention: null cu_q or tree");
    if (reinterpret_cast<uintptr_t>(tree) & 7u)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_tree_attention: tree must be 8-byte aligned");
    if (tree_words <= 0 || (long long)tree_words * 64 < max_draft_tokens)
        return pkv::set_error(PF_ERR_INVALID, "pf_paged_tree_attention: tree_words holds no max_draft_tokens bits");
    pkv::AttnMask mask;
    mask.kind = pkv::kMaskTree;
    mask.tree = tree;
    mask.tree_words = tree_words;
    return masked_call(pool, layer, q, block_tables, max_blocks_per_seq, context_lens, cu_q, n_seqs, max_draft_tokens,
                       n_q_heads, scale, mask, out, out_dtype, workspace, ws_bytes, fn, stream);
}

int pf_device_status(int *status_out, int reset, void *stream) {
    pkv::clear_error();
    if (!status_out) return pkv::set_error(PF_ERR_INVALID, "pf_device_status: status_out is null");
    int *dev = pkv::device_status_ptr();
    if (!dev) return PF_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int host = 0;
    cudaError_t e = cudaMemcpyAsync(&host, dev, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return pkv::cuda_error(e, "pf_device_status: read");
    *status_out = host;
    if (reset) {
        e = cudaMemsetAsync(dev, 0, sizeof(int), s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return pkv::cuda_error(e, "pf_device_status: reset");
    }
    return PF_OK;
}

}  // extern "C"

namespace pkv {

int decode_on_scratch(const pf_pool *pool, int layer, const void *q, const int32_t *block_tables, int max_blocks,
                      const int32_t *context_lens, int n_seqs, int n_q_heads, float scale, void *out, int out_dtype,
                      int split_tokens, void *scratch, size_t bytes, void *stream) {
    return decode_call(pool, layer, q, nullptr, nullptr, false, block_tables, max_blocks, context_lens, n_seqs,
                       n_q_heads, scale, out, out_dtype, split_tokens, scratch, bytes, stream, true);
}

}  // namespace pkv
