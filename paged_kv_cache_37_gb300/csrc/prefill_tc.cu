// prefill_tc.cu -- host side of prefill_tc.cuh: tensor maps, how contexts are
// cut, the launches; and the instances without a mask.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>

#include "prefill_tc.cuh"

namespace pkv {
namespace prefill_tc {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// K or V viewed as (64 elements, rows, halves, kv-heads) with strides (row,
// 128 bytes, head): a box {64, box_rows, 1, 1} is one 64-element half of
// box_rows consecutive rows of one kv-head, landing as [box_rows][128 bytes]
// in the 128-byte swizzle.
int encode(CUtensorMap *map, void *base, const pf_pool *pool, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return set_error(PF_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t rows = (cuuint64_t)pool->n_layers * pool->n_blocks * pool->block_size;
    const cuuint64_t D = (cuuint64_t)pool->head_dim;
    const cuuint64_t H = (cuuint64_t)pool->n_kv_heads;
    cuuint64_t dims[4] = {64, rows, D / 64, H};
    cuuint64_t strides[3] = {H * D * 2, 128, D * 2};
    cuuint32_t box[4] = {64u, (cuuint32_t)box_rows, 1u, 1u};
    cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(PF_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r));
    return PF_OK;
}

template <int D, bool SPLIT>
Kernels pick(bool causal, bool q8) {
    const MergeFn merge = causal ? merge_parts_kernel<D, true, kMaskNone> : merge_parts_kernel<D, false, kMaskNone>;
    if (q8) return {causal ? prefill_tc_kernel<D, true, true, SPLIT, kMaskNone> : prefill_tc_kernel<D, false, true, SPLIT, kMaskNone>, merge};
    if constexpr (SPLIT) return {prefill_tc_kernel<D, false, false, true, kMaskNone>, merge};   // (causal fp16 contexts are not cut)
    else return {causal ? prefill_tc_kernel<D, true, false, false, kMaskNone> : prefill_tc_kernel<D, false, false, false, kMaskNone>, merge};
}

Kernels kernels_for(int D, bool causal, bool q8, bool split, int mask) {
    if (mask == kMaskWindow) return window_kernels(D, q8, split);
    if (mask == kMaskTree) return tree_kernels(D, q8, split);
    if (D == 64) return split ? pick<64, true>(causal, q8) : pick<64, false>(causal, q8);
    return split ? pick<128, true>(causal, q8) : pick<128, false>(causal, q8);
}

// Workspace of a block's part.
size_t part_bytes(int D) { return (size_t)(2 * QT) * (D + 2) * sizeof(float); }

long long blocks_of(const pf_pool *pool, int n_seqs, int n_q_heads, int max_new) {
    return (long long)n_seqs * pool->n_kv_heads *
           (((long long)max_new * (n_q_heads / pool->n_kv_heads) + 2 * QT - 1) / (2 * QT));
}

}  // namespace
}  // namespace prefill_tc

// Parts that contexts are cut into: as many as give every SM a block, of at
// least kMinTiles tiles at the table's longest context, if that pays.  In
// microseconds a tile takes 0.9; the second launch 4, and the parts' way
// through L2 their bytes at 5 TB/s.  (Measured uncut / cut, 8 kv-heads: fp16 x
// 64, 32 rows, 4 x 2048 tokens 19.8 / 13.7, 1 x 65,536 tokens 456 / 37; 1 x 1024
// tokens 12.0 / 13.0; e4m3 x 128, 32 rows, 4 x 8192 tokens 115 / 37; 512 rows, 4
// x 2048 tokens 36.2 / 29.9, 4 x 1024 tokens 21.6 / 22.7.)
int prompt_splits(const pf_pool *pool, bool causal, int n_seqs, int n_q_heads, int max_blocks, int max_new, int sms,
                  size_t ws_bytes, const AttnMask &mask) {
    const long long blocks = prefill_tc::blocks_of(pool, n_seqs, n_q_heads, max_new);
    if ((causal && mask.kind == kMaskNone && pool->dtype == PF_F16) || blocks <= 0) return 1;
    const int BN = pool->head_dim == 64 ? prefill_tc::Cfg<64, false>::BN : prefill_tc::Cfg<128, false>::BN;
    long long tiles = ((long long)max_blocks * pool->block_size + BN - 1) / BN;
    if (mask.kind == kMaskWindow) {   // of a block: its sinks, and its rows' windows
        const long long tokens = std::min<long long>(max_new, 2 * prefill_tc::QT / (n_q_heads / pool->n_kv_heads) + 1);
        tiles = std::min(tiles, (mask.sinks + BN - 1ll) / BN + (mask.window + tokens + BN - 1ll) / BN + 1);
    }
    const long long room = ws_bytes < kWorkspaceFront ? 0 : (long long)((ws_bytes - kWorkspaceFront) / prefill_tc::part_bytes(pool->head_dim));   // parts that fit
    const long long n = std::min(std::min(std::min((long long)sms, room) / blocks, tiles / prefill_tc::kMinTiles),
                                 (long long)prefill_tc::kMaxParts);
    if (n < 2) return 1;
    const long long rows = std::min((long long)max_new * (n_q_heads / pool->n_kv_heads), 2ll * prefill_tc::QT);
    const double bytes = 2.0 * (double)(blocks * n * rows) * pool->head_dim * sizeof(float);
    return 0.9 * (double)(tiles - (tiles + n - 1) / n) > 4.0 + bytes / 5e6 ? (int)n : 1;
}

size_t prompt_workspace_bytes(const pf_pool *pool, bool causal, int n_seqs, int n_q_heads, int max_blocks, int max_new,
                              const AttnMask &mask) {
    int sms = 0;
    if (n_seqs <= 0 || max_new <= 0 || n_q_heads <= 0 || n_q_heads % pool->n_kv_heads || max_blocks <= 0 ||
        device_sms(false, &sms) != PF_OK)
        return 0;
    // a part per SM, whatever the batch: a smaller one takes no more
    return prompt_splits(pool, causal, n_seqs, n_q_heads, max_blocks, max_new, sms, SIZE_MAX, mask) == 1
               ? 0
               : kWorkspaceFront + sms * prefill_tc::part_bytes(pool->head_dim);
}

int launch_prefill_tc(const PrefillArgs &a, cudaStream_t stream) {
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    pf_pool *pool = const_cast<pf_pool *>(a.pool);
    const int D = pool->head_dim;
    const bool q8 = pool->dtype == PF_E4M3;
    const int BN = D == 64 ? prefill_tc::Cfg<64, false>::BN : prefill_tc::Cfg<128, false>::BN;
    const int gh = a.n_q_heads / pool->n_kv_heads;
    const long long n_items = (long long)a.n_seqs * pool->n_kv_heads;
    const long long n_qp = ((long long)a.max_new * gh + 2 * prefill_tc::QT - 1) / (2 * prefill_tc::QT);
    if (n_items * n_qp > 0x7fffffffll)
        return set_error(PF_ERR_INVALID, "pf_paged_prefill_attention: too many query tiles for one launch");
    const int box_rows = pool->block_size >= 16 ? (pool->block_size < BN ? pool->block_size : BN) : 1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "pf_paged_prefill_attention: cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return set_error(PF_ERR_UNSUPPORTED, "device index out of range");
    if (!q8) {   // e4m3 tiles are not copied by TMA
        std::lock_guard<std::mutex> lock(pool->mu);
        if (!pool->tmap_pf_ready[dev]) {
            int rc = prefill_tc::encode(&pool->tmap_pf_k[dev], pool->k_base, pool, box_rows);
            if (rc) return rc;
            rc = prefill_tc::encode(&pool->tmap_pf_v[dev], pool->v_base, pool, box_rows);
            if (rc) return rc;
            pool->tmap_pf_ready[dev] = true;
        }
    }
    prefill_tc::Params p;
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
    p.box_rows = box_rows;
    p.n_seqs = a.n_seqs;
    p.n_items = (int)n_items;
    p.n_qp = (int)n_qp;
    p.layer_page0 = (long long)a.layer * pool->n_blocks;
    p.layer_row0 = p.layer_page0 * pool->block_size;
    p.out_f32 = a.out_dtype == PF_F32;
    p.mask = a.mask;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.splits = 1;
    p.part_ml = nullptr;
    p.part_o = nullptr;
    const long long blocks = n_items * n_qp;
    if (a.workspace) {
        int sms = 0;
        const int rc = device_sms(true, &sms);
        if (rc) return rc;
        p.splits = prompt_splits(pool, a.causal, a.n_seqs, a.n_q_heads, a.max_blocks, a.max_new, sms, a.ws_bytes, a.mask);
        p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.workspace) + kWorkspaceFront);
        p.part_o = reinterpret_cast<float *>(p.part_ml + (size_t)blocks * p.splits * 2 * prefill_tc::QT);
    }
    const bool split = p.splits > 1;
    const prefill_tc::Kernels kernels = prefill_tc::kernels_for(D, a.causal, q8, split, a.mask.kind);
    const prefill_tc::KernelFn fn = kernels.main;
    const int smem = D == 64 ? (q8 ? prefill_tc::Cfg<64, true>::SMEM : prefill_tc::Cfg<64, false>::SMEM)
                             : (q8 ? prefill_tc::Cfg<128, true>::SMEM : prefill_tc::Cfg<128, false>::SMEM);
    // once per device and kernel (setting it twice does no harm)
    static std::atomic<bool> ready[kMaxDevices][3][16];
    std::atomic<bool> &done = ready[dev][a.mask.kind][(D == 64) + 2 * a.causal + 4 * q8 + 8 * split];
    if (!done.load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_error(e, "pf_paged_prefill_attention: cudaFuncSetAttribute");
        done.store(true, std::memory_order_release);
    }
    fn<<<(unsigned)(blocks * p.splits), prefill_tc::NTHREADS, smem, stream>>>(pool->tmap_pf_k[dev],
                                                                              pool->tmap_pf_v[dev], p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "pf_paged_prefill_attention: launch");
    if (split) {
        cudaLaunchConfig_t cfg = {};
        const long long most = std::min((long long)a.max_new * gh, 2ll * prefill_tc::QT);   // rows of a block
        cfg.gridDim = dim3((unsigned)blocks, (unsigned)((most + prefill_tc::kMergeWarps - 1) / prefill_tc::kMergeWarps));
        cfg.blockDim = dim3(32 * prefill_tc::kMergeWarps);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kernels.merge, p);
        if (e != cudaSuccess) return cuda_error(e, "pf_paged_prefill_attention: merge launch");
    }
    return PF_OK;
}

}  // namespace pkv
