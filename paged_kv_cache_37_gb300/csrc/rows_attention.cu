// rows_attention.cu -- host side of rows_attention.cuh: the partition's grid,
// the workspace and the launches.
#include <mutex>

#include "rows_attention.cuh"

namespace pkv {
namespace {

// SMs assumed when no device can be queried (sizes a workspace only).
constexpr int kSmsNoDevice = 256;
constexpr size_t kReserved = 256;   // front of every workspace, unused here

// Warps per team: as many as 4 of the kv-heads, spread evenly over the groups
// (5 heads: 3 + 2, so that one warp in six idles instead of three in eight).
int heads_per_team(int n_kv_heads) {
    const int groups = (n_kv_heads + 3) / 4;
    return (n_kv_heads + groups - 1) / groups;
}

rows::Kernel kernel_for(const pf_pool *pool, int n_rows, bool f32) {
    return pool->dtype == PF_E4M3 ? rows::kernel_e4m3(pool->head_dim, n_rows, f32)
                                  : rows::kernel_f16(pool->head_dim, n_rows, f32);
}

}  // namespace

int rows_plan(const pf_pool *pool, int n_rows, bool need_device, RowsPlan *plan) {
    int sms = 0, dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (need_device) return cuda_error(e, "attention: SM count");
        sms = kSmsNoDevice;
    }
    plan->grid = sms;
    const int hg = heads_per_team(pool->n_kv_heads);
    const size_t warps = (size_t)sms * (rows::NW / hg) * hg;
    plan->counter_bytes = (warps * sizeof(unsigned long long) + 255) / 256 * 256;
    plan->bytes = kReserved + plan->counter_bytes +
                  warps * 2 * (size_t)n_rows * (size_t)(pool->head_dim + 4) * sizeof(float);
    return PF_OK;
}

int launch_rows(const RowsArgs &a, cudaStream_t stream) {
    const pf_pool *pool = a.pool;
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    const rows::Kernel k = kernel_for(pool, a.rows, a.out_dtype == PF_F32);
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(k.fn),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e != cudaSuccess) return cuda_error(e, "attention: cudaFuncSetAttribute");
    rows::Params p;
    p.k_pool = static_cast<const uint8_t *>(pool->k_base);
    p.v_pool = static_cast<const uint8_t *>(pool->v_base);
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.status = status;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace) + kReserved;
    p.counters = reinterpret_cast<unsigned long long *>(ws);
    p.recs = reinterpret_cast<float *>(ws + a.plan.counter_bytes);
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
    p.scale_log2 = a.scale * 1.4426950408889634f;
    const size_t row = (size_t)a.n_q_heads * pool->head_dim;
    const size_t out_elem = a.out_dtype == PF_F32 ? 4 : 2;
    // Sequences are independent: larger batches are consecutive launches.
    for (int s0 = 0; s0 < a.n_seqs; s0 += rows::kMaxSeqs) {
        const size_t q0 = a.cu_q ? 0 : (size_t)s0 * row;   // cu_q holds absolute rows
        p.q = static_cast<const __half *>(a.q) + q0;
        p.out = static_cast<uint8_t *>(a.out) + q0 * out_elem;
        p.bt = a.block_tables + (size_t)s0 * a.max_blocks;
        p.lens = a.context_lens + s0;
        p.cu_q = a.cu_q ? a.cu_q + s0 : nullptr;
        p.n_seqs = a.n_seqs - s0 < rows::kMaxSeqs ? a.n_seqs - s0 : rows::kMaxSeqs;
        p.epoch = next_epoch();
        k.fn<<<(unsigned)a.plan.grid, rows::NTHREADS, k.smem, stream>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_error(e, "attention: launch");
    }
    return PF_OK;
}

}  // namespace pkv
