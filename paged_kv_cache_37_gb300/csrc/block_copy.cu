// block_copy.cu -- whole-block copies: copy-on-write copies inside the pool
// (pf_copy_blocks) and swapping blocks to and from host memory (pf_swap_out,
// pf_swap_in).
//
// A block of one layer is B * Hkv * D fp16 values, contiguous in the pool
// (PageForge, "Four layers, one pointer": one page holds all heads of its
// tokens).  A copy-on-write gives a diverging sequence its own copy of a
// shared block in every layer (PagedAttention blog, "Copy-on-Write for
// Parallel Sampling"); swapping moves a block's contents, every layer, K and
// V, to CPU memory and back (same blog, "Preemption and Swapping").  The host
// side is a sequence of block images [n_layers][2][B][Hkv][D].
//
// One CTA moves one (block, layer, K or V) with 16-byte vectors, several in
// flight per thread.  For swapping, the kernel reads or writes the
// page-locked host buffer directly through its device mapping (on GB300 the
// Grace memory is reached over NVLink-C2C), so no staging buffer and no
// per-block memcpy is needed.  Pure copies: bit-exact.
//
// e4m3 pools: a block of one layer is B * Hkv * D codes and Hkv fp32 scales
// (K's and V's each); an image holds them one after the other, the scales
// padded to 16 bytes.
//
// Compaction (pf_compact_blocks) is the same copy -- no destination is a
// source -- with the block tables' used entries sent through the block map by
// further CTAs of the launch: the copy does not read the tables.  HBM bound:
// 229 MB read and written over 12 layers take 36.3 us, 6.31 TB/s (GB300).
#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // 16-byte vectors in flight per thread

struct BlockCopyParams {
    // pool bases, or (when the ids on that side are null) the image array in
    // the *_k pointer
    const uint4 *src_k;
    const uint4 *src_v;
    uint4 *dst_k;
    uint4 *dst_v;
    const int32_t *src_ids;   // null: source i is image i
    const int32_t *dst_ids;   // null: destination i is image i
    int *status;
    int n_layers;
    int n_blocks;
    int64_t vecs;             // 16-byte vectors per block of one layer
    // e4m3 pools: scales [layer][block][heads] (in an image they follow the codes)
    const float *k_scale;
    const float *v_scale;
    int heads;                // scales per block of one layer (fp16 pools: 0)
    int64_t image_vecs;       // vecs, and the scales padded to whole vectors
    // compaction
    int n_copies;
    const int32_t *map;
    int32_t *tables;
    const int32_t *lens;
    int n_rows;
    int max_blocks;
    int block_size;
};

// Table entries that a context uses, through the map (CTA `part` of `parts`).
__device__ __forceinline__ void remap_tables(const BlockCopyParams &p, int part, int parts) {
    const int64_t total = (int64_t)p.n_rows * p.max_blocks;
    for (int64_t e = (int64_t)part * kThreads + threadIdx.x; e < total; e += (int64_t)parts * kThreads) {
        const int s = (int)(e / p.max_blocks);
        const int64_t tok = (e - (int64_t)s * p.max_blocks) * p.block_size;
        int64_t L = p.lens[s];
        const int64_t most = (int64_t)p.max_blocks * p.block_size;
        if (L < 0 || L > most) {
            atomicOr(p.status, PF_DEV_BAD_LENGTH);
            L = L < 0 ? 0 : most;
        }
        if (tok >= L) continue;
        const int id = p.tables[e];
        const int to = id >= 0 && id < p.n_blocks ? p.map[id] : -1;
        if (to < 0 || to >= p.n_blocks) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);   // the entry stays
        else if (to != id) p.tables[e] = to;
    }
}

// Address of (item i, layer, kv) on one side, or null for a bad block id.
__device__ __forceinline__ const uint4 *side_addr(const uint4 *pool_k, const uint4 *pool_v, const int32_t *ids,
                                                  int i, int layer, int kv, const BlockCopyParams &p) {
    if (ids == nullptr) return pool_k + (((int64_t)i * p.n_layers + layer) * 2 + kv) * p.image_vecs;
    const int b = ids[i];
    if (b < 0 || b >= p.n_blocks) return nullptr;
    return (kv ? pool_v : pool_k) + ((int64_t)layer * p.n_blocks + b) * p.vecs;
}

__global__ void __launch_bounds__(kThreads) block_copy_kernel(const BlockCopyParams p) {
    const int i = blockIdx.x;
    if (i >= p.n_copies) {
        if (blockIdx.y == 0) remap_tables(p, i - p.n_copies, gridDim.x - p.n_copies);
        return;
    }
    const int layer = blockIdx.y >> 1;
    const int kv = blockIdx.y & 1;
    const uint4 *src = side_addr(p.src_k, p.src_v, p.src_ids, i, layer, kv, p);
    uint4 *dst = const_cast<uint4 *>(side_addr(p.dst_k, p.dst_v, p.dst_ids, i, layer, kv, p));
    if (src == nullptr || dst == nullptr) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
        return;   // the pair is skipped in every layer
    }
    if (p.heads) {
        const float *s = p.src_ids ? (kv ? p.v_scale : p.k_scale) + ((int64_t)layer * p.n_blocks + p.src_ids[i]) * p.heads
                                   : reinterpret_cast<const float *>(src + p.vecs);
        float *d = p.dst_ids ? const_cast<float *>(kv ? p.v_scale : p.k_scale) +
                                  ((int64_t)layer * p.n_blocks + p.dst_ids[i]) * p.heads
                             : reinterpret_cast<float *>(dst + p.vecs);
        for (int h = threadIdx.x; h < p.heads; h += kThreads) d[h] = s[h];
    }
    for (int64_t v0 = threadIdx.x; v0 < p.vecs; v0 += (int64_t)kThreads * kUnroll) {
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + (int64_t)u * kThreads;
            if (v < p.vecs) x[u] = ld_stream(src + v);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + (int64_t)u * kThreads;
            if (v < p.vecs) st_stream(dst + v, x[u]);
        }
    }
}

}  // namespace

int launch_block_copy(const BlockCopyArgs &a, cudaStream_t stream) {
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    const pf_pool *pool = a.pool;
    if (pool->n_layers > 65535 / 2) return set_error(PF_ERR_INVALID, "block copy: too many layers for one launch");
    BlockCopyParams p;
    const uint4 *pk = static_cast<const uint4 *>(pool->k_base);
    const uint4 *pv = static_cast<const uint4 *>(pool->v_base);
    if (a.src_ids) {
        p.src_k = pk;
        p.src_v = pv;
    } else {
        p.src_k = static_cast<const uint4 *>(a.image);
        p.src_v = nullptr;
    }
    if (a.dst_ids) {
        p.dst_k = const_cast<uint4 *>(pk);
        p.dst_v = const_cast<uint4 *>(pv);
    } else {
        p.dst_k = static_cast<uint4 *>(const_cast<void *>(a.image));
        p.dst_v = nullptr;
    }
    p.src_ids = a.src_ids;
    p.dst_ids = a.dst_ids;
    p.status = status;
    p.n_layers = pool->n_layers;
    p.n_blocks = pool->n_blocks;
    const bool q8 = pool->dtype == PF_E4M3;
    p.vecs = (int64_t)pool->block_size * pool->n_kv_heads * pool->head_dim / (q8 ? 16 : 8);
    p.heads = q8 ? pool->n_kv_heads : 0;
    p.image_vecs = p.vecs + (p.heads + 3) / 4;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.n_copies = a.n;
    p.map = a.block_map;
    p.tables = a.block_tables;
    p.lens = a.context_lens;
    p.n_rows = a.n_rows;
    p.max_blocks = a.max_blocks;
    p.block_size = pool->block_size;
    const int64_t entries = a.block_tables ? (int64_t)a.n_rows * a.max_blocks : 0;
    const int64_t remap = (entries + 4 * kThreads - 1) / (4 * kThreads);   // four entries per thread
    const int64_t grid_x = a.n + (remap < 4096 ? remap : 4096);
    if (grid_x > 0x7fffffffll) return set_error(PF_ERR_INVALID, "block copy: too many blocks for one launch");
    dim3 grid((unsigned)grid_x, (unsigned)(pool->n_layers * 2));
    block_copy_kernel<<<grid, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "block copy: launch");
    return PF_OK;
}

}  // namespace pkv
