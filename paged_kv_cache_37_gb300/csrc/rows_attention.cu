// rows_attention.cu -- host side of rows_attention.cuh: the partition's grid,
// the workspace and the launches.
#include <algorithm>
#include <atomic>

#include "rows_attention.cuh"

namespace pkv {
namespace {

// SMs assumed when no device can be queried (sizes a workspace only).
constexpr int kSmsNoDevice = 256;

// Warps per team: as many as 4 of the kv-heads, spread evenly over the groups
// (5 heads: 3 + 2, so that one warp in six idles instead of three in eight).
int heads_per_team(int n_kv_heads) {
    const int groups = (n_kv_heads + 3) / 4;
    return (n_kv_heads + groups - 1) / groups;
}

rows::Kernel kernel_for(const pf_pool *pool, int n_rows, bool f32, int mask) {
    const bool paged = pool->block_size >= 16;
    const bool d64 = pool->head_dim == 64;
    const bool q8 = pool->dtype == PF_E4M3;
    if (mask == kMaskWindow)
        return q8 ? (d64 ? rows::kernel_e4m3_d64_window : rows::kernel_e4m3_d128_window)(n_rows, f32, paged)
                  : (d64 ? rows::kernel_f16_d64_window : rows::kernel_f16_d128_window)(n_rows, f32, paged);
    if (mask == kMaskTree)
        return q8 ? (d64 ? rows::kernel_e4m3_d64_tree : rows::kernel_e4m3_d128_tree)(n_rows, f32, paged)
                  : (d64 ? rows::kernel_f16_d64_tree : rows::kernel_f16_d128_tree)(n_rows, f32, paged);
    return q8 ? (d64 ? rows::kernel_e4m3_d64 : rows::kernel_e4m3_d128)(n_rows, f32, paged)
              : (d64 ? rows::kernel_f16_d64 : rows::kernel_f16_d128)(n_rows, f32, paged);
}

}  // namespace

int device_sms(bool need_device, int *out) {
    static std::atomic<int> known[kMaxDevices];   // SMs per device, 0: not asked yet
    int sms = 0, dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) sms = known[dev].load(std::memory_order_relaxed);
    if (e == cudaSuccess && sms == 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) known[dev].store(sms, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (need_device) return cuda_error(e, "attention: SM count");
        sms = kSmsNoDevice;
    }
    *out = sms;
    return PF_OK;
}

int rows_plan(const pf_pool *pool, int n_rows, bool need_device, RowsPlan *plan, size_t most) {
    int sms = 0;
    const int rc = device_sms(need_device, &sms);
    if (rc) return rc;
    plan->sms = sms;
    const int hg = heads_per_team(pool->n_kv_heads);
    const size_t warps = (size_t)(kernel_for(pool, n_rows, false, kMaskNone).warps / hg) * hg;   // of a CTA
    const size_t recs = warps * 2 * (size_t)n_rows * (size_t)(pool->head_dim + 4) * sizeof(float);
    const size_t room = (most < kWorkspaceFront ? 0 : most - kWorkspaceFront) / recs;
    plan->grid = (int)std::min(room, (size_t)std::min(sms, kFlagSms));
    if (plan->grid == 0) return set_error(PF_ERR_INVALID, "attention: the scratch holds no block's records");
    plan->bytes = kWorkspaceFront + plan->grid * recs;
    return PF_OK;
}

int launch_rows(const RowsArgs &a, cudaStream_t stream) {
    const pf_pool *pool = a.pool;
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    const rows::Kernel k = kernel_for(pool, a.rows, a.out_dtype == PF_F32, a.mask.kind);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "attention: cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return set_error(PF_ERR_UNSUPPORTED, "device index out of range");
    // once per device and kernel (setting it twice does no harm)
    static std::atomic<bool> ready[kMaxDevices][3][32];
    std::atomic<bool> &done = ready[dev][a.mask.kind][(pool->dtype == PF_E4M3) + 2 * (pool->head_dim == 64) + 4 * (a.rows <= 8) +
                                         8 * (a.out_dtype == PF_F32) + 16 * (pool->block_size >= 16)];
    if (!done.load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(k.fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 k.smem);
        if (e != cudaSuccess) return cuda_error(e, "attention: cudaFuncSetAttribute");
        done.store(true, std::memory_order_release);
    }
    rows::Params p;
    p.k_pool = static_cast<const uint8_t *>(pool->k_base);
    p.v_pool = static_cast<const uint8_t *>(pool->v_base);
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.status = status;
    p.flags = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(a.workspace) + kFlagOffset);
    p.recs = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kWorkspaceFront);
    p.max_blocks = a.max_blocks;
    p.n_blocks = pool->n_blocks;
    p.block_size = pool->block_size;
    p.block_shift = 0;
    while ((1 << p.block_shift) < pool->block_size) ++p.block_shift;
    p.n_q_heads = a.n_q_heads;
    p.n_kv_heads = pool->n_kv_heads;
    p.gh = a.n_q_heads / pool->n_kv_heads;
    p.hg = heads_per_team(pool->n_kv_heads);
    p.n_groups = (pool->n_kv_heads + p.hg - 1) / p.hg;
    p.rows = a.rows;
    p.causal = a.causal ? 1 : 0;
    p.out_f32 = a.out_dtype == PF_F32;
    p.layer_page0 = (long long)a.layer * pool->n_blocks;
    p.layer_row0 = p.layer_page0 * pool->block_size;
    p.mask = a.mask;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    const size_t row = (size_t)a.n_q_heads * pool->head_dim;
    const size_t out_elem = a.out_dtype == PF_F32 ? 4 : 2;
    // Sequences are independent: larger batches are consecutive launches, of
    // as many as keep the work units below 2^31 however long the contexts are.
    const long long most = ((long long)a.max_blocks * pool->block_size / 16 + 1 + rows::kPairCost) * p.n_groups;
    if (most > 0x7fffffffll) return set_error(PF_ERR_INVALID, "attention: max_blocks_per_seq is too large for the heads");
    bool captured = false;
    const int rc = is_captured(stream, &captured);
    if (rc) return rc;
    const int step = (int)(0x7fffffffll / most < rows::kMaxSeqs ? 0x7fffffffll / most : rows::kMaxSeqs);
    for (int s0 = 0; s0 < a.n_seqs; s0 += step) {
        const size_t q0 = a.cu_q ? 0 : (size_t)s0 * row;   // cu_q holds absolute rows
        p.q = static_cast<const __half *>(a.q) + q0;
        p.out = static_cast<uint8_t *>(a.out) + q0 * out_elem;
        p.bt = a.block_tables + (size_t)s0 * a.max_blocks;
        p.lens = a.context_lens + s0;
        p.cu_q = a.cu_q ? a.cu_q + s0 : nullptr;
        p.n_seqs = a.n_seqs - s0 < step ? a.n_seqs - s0 : step;
        p.stamp = captured ? 0 : host_stamp(next_epoch());
        p.after_append = a.after_append && s0 == 0;
        // a programmatic dependent of the kernel before it: its blocks take
        // their SMs as that kernel's leave them, and then wait for its end
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)a.plan.grid);
        cfg.blockDim = dim3((unsigned)k.warps * 32);
        cfg.dynamicSmemBytes = (size_t)k.smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, k.fn, p);
        if (e != cudaSuccess) return cuda_error(e, "attention: launch");
    }
    return PF_OK;
}

}  // namespace pkv
