// prompt_masked.cu -- host side of prompt_masked.cuh: how contexts are cut, the
// workspace and the launches.
#include <algorithm>
#include <atomic>

#include "prompt_masked.cuh"

namespace pkv {
namespace {

int tile_tokens(const pf_pool *pool) {
    return pool->head_dim == 64 ? prompt_masked::Cfg<64, false, false>::BN : prompt_masked::Cfg<128, false, false>::BN;
}

// Rows that are looked up and copied together (the TMA boxes of fp16 pools): 16 of
// e4m3 pages and under windows, whose blocks walk whole boxes from their first token
// on, otherwise what a page holds of a tile.  Boxes of 16 / 64 rows of pages of 64: 4
// prompts of 4,096 tokens, window 512, 32 q-heads over 8 kv-heads x 128 142 / 154 us.  With
// one query tile a block (dual; 30 rows x 4, 8 kv-heads) it depends on more than the
// window: x 128, 2 sequences, not cut, window 512 11.9 / 12.1, 768 14.2 / 14.2, 1,024
// 16.8 / 16.5, 2,048 26.5 / 25.1, 4,000 45.2 / 41.3; but 64 sequences, window 256 28.8 /
// 35.2, 512 41.2 / 46.3, 1,024 64.1 / 67.6, 2,048 107.5 / 109.1; x 64 within 2 % over
// pages of 64, over pages of 256 (boxes of 128) 64 sequences, window 512 30.4 / 37.0, 2,048
// 65.8 / 69.7.  The border serves the uncut calls of few blocks.
constexpr int kSmallBoxWindow = 512;
int unit_rows(const pf_pool *pool, const AttnMask &mask, bool dual) {
    if (pool->block_size < 16) return 1;
    if (pool->dtype == PF_E4M3 || (mask.kind == kMaskWindow && !(dual && mask.window > kSmallBoxWindow))) return 16;
    return std::min(pool->block_size, tile_tokens(pool));
}

// Tokens that a block sees at most: the table's, or a window's (its sinks, and its
// rows' windows), in whole boxes.
long long block_tokens(const pf_pool *pool, const AttnMask &mask, int n_q_heads, int max_blocks, int max_new) {
    const long long group = n_q_heads / pool->n_kv_heads, tokens = (long long)max_blocks * pool->block_size;
    if (mask.kind != kMaskWindow) return tokens;
    return std::min(tokens, (long long)mask.sinks + mask.window + std::min<long long>(max_new, prompt_masked::ROWS / group + 1) +
                                2 * unit_rows(pool, mask, max_new * group <= prompt_masked::QT));
}

// Workspace of a block's part.
size_t part_bytes(const pf_pool *pool) {
    return (size_t)prompt_masked::ROWS * (pool->head_dim + 2) * sizeof(float);
}

}  // namespace

// Parts that contexts are cut into: as many as give every SM a block, of at
// least kMinTiles tiles at the table's longest context (a window's), if that
// pays: 0.9 us a tile saved against 4 us for the second launch and the parts'
// bytes.  Uncut -> cut, trees over fp16 x 128: 8 blocks of 128 rows, 1,024 tokens
// 15.0 -> 12.2 us, 4,096 42.2 -> 13.2; 64 blocks of 256 rows 1,024 tokens 19.2 ->
// 22.6 (not taken), 2,048 31.9 -> 30.1.  A tile takes from 0.56 us (fp16 x 128, one
// query tile) to 1.24 (fp16 x 64, two); with 0.9 for all of them the choice costs 0.4 %
// on average and 1.9 us at most (e4m3 x 64, 8 blocks of 1,024 tokens, 15.2 cut, 17.1
// as chosen) over 152 cases: both types and head_dims, 30 to 250 drafts x 4 of 1 to 8
// sequences, 8 kv-heads, 512 to 8,192 tokens.
int masked_splits(const pf_pool *pool, const AttnMask &mask, int n_seqs, int n_q_heads, int max_blocks, int max_new,
                  int sms, size_t ws_bytes) {
    const long long group = n_q_heads / pool->n_kv_heads, all_rows = max_new * group;
    const long long blocks = (long long)n_seqs * pool->n_kv_heads * ((all_rows + prompt_masked::ROWS - 1) / prompt_masked::ROWS);
    if (blocks <= 0) return 1;
    const long long tiles = (block_tokens(pool, mask, n_q_heads, max_blocks, max_new) + tile_tokens(pool) - 1) / tile_tokens(pool);
    const long long room = ws_bytes < kWorkspaceFront ? 0 : (long long)((ws_bytes - kWorkspaceFront) / part_bytes(pool));
    const long long n = std::min(std::min(std::min((long long)sms, room) / blocks, tiles / prompt_masked::kMinTiles),
                                 (long long)prompt_masked::kMaxParts);
    if (n < 2) return 1;
    const double bytes = 2.0 * (double)(blocks * n * std::min<long long>(all_rows, prompt_masked::ROWS)) * pool->head_dim * sizeof(float);
    return 0.9 * (double)(tiles - (tiles + n - 1) / n) > 4.0 + bytes / 5e6 ? (int)n : 1;
}

size_t masked_workspace_bytes(const pf_pool *pool, const AttnMask &mask, int n_seqs, int n_q_heads, int max_blocks, int max_new) {
    int sms = 0;
    if (n_seqs <= 0 || max_new <= 0 || n_q_heads <= 0 || n_q_heads % pool->n_kv_heads || max_blocks <= 0 ||
        device_sms(false, &sms) != PF_OK)
        return 0;
    // a part per SM, whatever the batch: a smaller one takes no more
    return masked_splits(pool, mask, n_seqs, n_q_heads, max_blocks, max_new, sms, SIZE_MAX) == 1
               ? 0
               : kWorkspaceFront + sms * part_bytes(pool);
}

int launch_prompt_masked(const PrefillArgs &a, cudaStream_t stream) {
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    pf_pool *pool = const_cast<pf_pool *>(a.pool);
    const int D = pool->head_dim;
    const bool q8 = pool->dtype == PF_E4M3;
    const int gh = a.n_q_heads / pool->n_kv_heads;
    const long long rows = (long long)a.max_new * gh;
    const long long n_items = (long long)a.n_seqs * pool->n_kv_heads;
    const long long n_qp = (rows + prompt_masked::ROWS - 1) / prompt_masked::ROWS;
    const long long blocks = n_items * n_qp;
    // One query tile a block: both softmax groups take its tiles, even and odd.  With
    // the second group idle instead, 32 sequences of 256 to 2,048 tokens, 8 kv-heads,
    // 12 to 32 drafts x 4 q-heads: x 64 28.9 us for 22.7, x 128 36.9 for 36.3, e4m3 x
    // 128 40.5 for 39.3.  (More rows need both query tiles.)
    const bool dual = rows <= prompt_masked::QT;
    if (blocks > 0x7fffffffll) return set_error(PF_ERR_INVALID, "attention: too many query tiles for one launch");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "attention: cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return set_error(PF_ERR_UNSUPPORTED, "device index out of range");
    int rc = device_sms(true, &sms);
    if (rc) return rc;
    const int unit = unit_rows(pool, a.mask, dual), boxes = unit == 16 ? 1 : 2;
    if (!q8 && (rc = encode_prompt_tmaps(pool, dev, boxes, unit)) != PF_OK) return rc;   // e4m3 tiles are not copied by TMA
    prompt_masked::Params p;
    p.q = static_cast<const __half *>(a.q);
    p.k_pool = pool->k_base;
    p.v_pool = pool->v_base;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.out = a.out;
    p.bt = a.block_tables;
    p.lens = a.context_lens;
    p.cu_q = a.cu_q;
    p.status = status;
    p.n_q_heads = a.n_q_heads;
    p.n_kv_heads = pool->n_kv_heads;
    p.gh = gh;
    p.gh_magic = (65536 + gh - 1) / gh;
    p.max_blocks = a.max_blocks;
    p.max_new = a.max_new;
    p.n_blocks = pool->n_blocks;
    p.block_size = pool->block_size;
    p.block_shift = 0;
    while ((1 << p.block_shift) < pool->block_size) ++p.block_shift;
    p.unit_shift = 0;
    while ((1 << p.unit_shift) < unit) ++p.unit_shift;
    p.n_seqs = a.n_seqs;
    p.n_items = (int)n_items;
    p.n_qp = (int)n_qp;
    p.layer_page0 = (long long)a.layer * pool->n_blocks;
    p.layer_row0 = p.layer_page0 * pool->block_size;
    p.out_f32 = a.out_dtype == PF_F32;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.mask = a.mask;
    p.splits = 1;
    p.part_ml = nullptr;
    p.part_o = nullptr;
    if (a.workspace) {
        p.splits = masked_splits(pool, a.mask, a.n_seqs, a.n_q_heads, a.max_blocks, a.max_new, sms, a.ws_bytes);
        p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.workspace) + kWorkspaceFront);
        p.part_o = reinterpret_cast<float *>(p.part_ml + (size_t)blocks * p.splits * prompt_masked::ROWS);
    }
    const bool split = p.splits > 1;
    p.n_work = (int)(blocks * p.splits);     // (cut: no more than SMs)
    const unsigned grid = (unsigned)std::min(p.n_work, sms);
    // A wait may last as long as kInfos + 1 blocks, and as long as all of a CTA's blocks
    // are looked at: beside what any wait has, 33 us for each tile of the longest (one
    // takes 0.3 to 2.5) and 0.13 us for each block (0.02).
    const long long most_tiles = block_tokens(pool, a.mask, a.n_q_heads, a.max_blocks, a.max_new) / tile_tokens(pool) + 1;
    p.wait_ns = kWaitLimitNs + ((unsigned long long)most_tiles << 15) + ((unsigned long long)(p.n_work / grid) << 7);
    const prompt_masked::Kernels k = a.mask.kind == kMaskWindow ? prompt_masked::window_kernels(D, q8, split, dual)
                                                                : prompt_masked::tree_kernels(D, q8, split, dual);
    // once per device and kernel (setting it twice does no harm)
    static std::atomic<bool> ready[kMaxDevices][32];
    std::atomic<bool> &done = ready[dev][(D == 64) + 2 * q8 + 4 * split + 8 * (a.mask.kind == kMaskWindow) + 16 * dual];
    if (!done.load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(k.main), cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
        if (e != cudaSuccess) return cuda_error(e, "attention: cudaFuncSetAttribute");
        done.store(true, std::memory_order_release);
    }
    k.main<<<grid, prompt_masked::NTHREADS, k.smem, stream>>>(pool->tmap_pf_k[dev][boxes], pool->tmap_pf_v[dev][boxes], p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "attention: launch");
    if (split) {
        cudaLaunchConfig_t cfg = {};
        const long long most = std::min<long long>(rows, prompt_masked::ROWS);   // rows of a block
        cfg.gridDim = dim3((unsigned)blocks, (unsigned)((most + prompt_masked::kMergeWarps - 1) / prompt_masked::kMergeWarps));
        cfg.blockDim = dim3(32 * prompt_masked::kMergeWarps);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, k.merge, p);
        if (e != cudaSuccess) return cuda_error(e, "attention: merge launch");
    }
    return PF_OK;
}

}  // namespace pkv
