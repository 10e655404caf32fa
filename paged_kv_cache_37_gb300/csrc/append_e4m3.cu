// append_e4m3.cu -- writing into and reading back from an 8-bit (e4m3) pool:
// the quantising append (pf_append_kv) and the gather that widens
// (pf_gather_kv on such a pool).
//
// Page p of kv-head h holds e4m3 codes and one scale, a power of two: row =
// code * scale.  An append gives a touched page
//   scale' = max(scale, 2^k),  k = the smallest integer >= -24 with
//                              max |x| <= 448 * 2^k over the new rows x,
// (only 2^k where no earlier token of the sequence lies in the page) and
// stores code = e4m3(x / scale'), nearest even, magnitudes at most
// min(448, 61440 / scale') so that a row read back is a finite fp16.  Where
// the scale grows, the page's earlier rows are rounded again to it.
// With powers of two x / scale' is exact, so a code is one rounding of x
// (half a step: 2^-4 relative), and growing a scale moves exponents only: it
// is lossless but for codes that fall below e4m3's smallest normal, 2^-6.
// Rows of inf or NaN are flagged; inf is stored as the largest magnitude, NaN
// as 0, and neither counts for the scale.
//
// Append: 2 bytes read and 1 written per value, HBM bound: 8192 tokens of 40
// heads x 128 take 40.4 us, 6.24 TB/s; one token each for 128 sequences 2.9 us,
// a launch and three dependent loads.  One group of
// threads takes one (page, kv-head, K or V) and keeps all its new rows in
// registers between the maximum and the rounding, so they are read once; the
// group is a warp for 16-token pages (4 or 8 16-byte loads in flight per
// lane), 8 or 16 lanes for 1-token pages, 2 to 8 warps above.
#include <algorithm>

#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr unsigned FULL = 0xffffffffu;

struct AppendParams {
    const __half *k_new;
    const __half *v_new;
    uint8_t *k_pool;
    uint8_t *v_pool;
    float *k_scale;
    float *v_scale;
    const int32_t *bt;
    const int32_t *lens;
    const int32_t *cu;
    int *status;
    int max_blocks;
    int max_new;
    int n_blocks;
    int n_kv_heads;
    int blocks_per_seq;      // CTAs of one sequence
    int max_pages;           // pages the new tokens of one sequence touch, at most
    long long layer_page0;   // layer * n_blocks
};

template <int B, int D>
struct AppendShape {
    static constexpr int CHUNKS = B * D / 8;                                     // 16-byte chunks of a page's head
    // threads of a group: 8 chunks each, at least a warp (below 32 chunks one each), at most the CTA
    static constexpr int GT = CHUNKS < 32 ? CHUNKS : (CHUNKS / 8 < 32 ? 32 : (CHUNKS / 8 > kThreads ? kThreads : CHUNKS / 8));
    static constexpr int VPT = CHUNKS / GT;
    static constexpr int GROUPS = kThreads / GT;
};

// Magnitudes of w's two halves, as fp16 bits (which order as integers).
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & 0x7fff7fffu; }

// The same with inf and NaN as 0.
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t w) {
    const uint32_t m = magnitudes(w);
    return ((m & 0xffffu) < 0x7c00u ? m & 0xffffu : 0u) | (m < 0x7c000000u ? m & 0xffff0000u : 0u);
}

// Two halves, times a power of two, to e4m3 codes.
__device__ __forceinline__ uint32_t scaled_e4m3x2(uint32_t w, __half2 by) {
    const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&w), by);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    return r;
}

template <int B, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    using S = AppendShape<B, D>;
    griddep_launch();   // the attention of a fused step sets out; it waits for this grid's end before it reads a page
    constexpr int CPR = D / 8;                     // chunks of a row
    __shared__ uint32_t warp_max[kThreads / 32];
    const int s = blockIdx.x / p.blocks_per_seq;
    const int group = threadIdx.x / S::GT, tg = threadIdx.x % S::GT;
    const int task = (int)(blockIdx.x % p.blocks_per_seq) * S::GROUPS + group;
    const int H = p.n_kv_heads;
    const int j = task / (2 * H);                  // page among those the new tokens touch
    const int kv = task % (2 * H) / H;
    const int h = task % H;

    int L = p.lens[s];
    const int most = p.max_blocks * B;
    const bool flagger = threadIdx.x == 0 && blockIdx.x % p.blocks_per_seq == 0;
    if (L < 0 || L > most) {
        if (flagger) atomicOr(p.status, PF_DEV_BAD_LENGTH);
        L = L < 0 ? 0 : most;
    }
    const int q0 = p.cu ? p.cu[s] : s;
    int n = p.cu ? p.cu[s + 1] - q0 : (L > 0 ? 1 : 0);
    if (n < 0 || n > L || n > p.max_new) {
        if (flagger) atomicOr(p.status, PF_DEV_BAD_LENGTH);
        n = n < 0 ? 0 : min(min(n, L), p.max_new);
    }
    const int start = L - n;
    const int page = start / B + j;
    bool live = n > 0 && j < p.max_pages && page < (L + B - 1) / B;
    int blk = 0;
    if (live) {
        blk = p.bt[(size_t)s * p.max_blocks + page];
        if (blk < 0 || blk >= p.n_blocks) {
            if (tg == 0) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
            live = false;
        }
    }
    const int lo = max(start - page * B, 0);       // new rows of the page: lo .. hi - 1
    const int hi = min(L - page * B, B);
    float *scale_at = (kv ? p.v_scale : p.k_scale) + (size_t)(p.layer_page0 + blk) * H + h;
    const float old = live && lo > 0 ? *scale_at : 0.0f;

    uint4 x[S::VPT];
    uint32_t top2 = 0;
    const __half *rows = (kv ? p.v_new : p.k_new) + ((ptrdiff_t)(q0 + page * B - start) * H + h) * D;   // the page's row 0, new or not
#pragma unroll
    for (int i = 0; i < S::VPT; ++i) {
        const int e = i * S::GT + tg;
        const int t = e / CPR, c = e % CPR;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (live && t >= lo && t < hi) x[i] = ld_stream(reinterpret_cast<const uint4 *>(rows + (ptrdiff_t)t * H * D + c * 8));
    }
#pragma unroll
    for (int i = 0; i < S::VPT; ++i)
        top2 = __vmaxu2(__vmaxu2(top2, __vmaxu2(magnitudes(x[i].x), magnitudes(x[i].y))),
                        __vmaxu2(magnitudes(x[i].z), magnitudes(x[i].w)));
    uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    const bool bad = top >= 0x7c00u;               // inf or NaN among this thread's values
    if (bad) {
        atomicOr(p.status, PF_DEV_NONFINITE);
        top2 = 0;
#pragma unroll
        for (int i = 0; i < S::VPT; ++i)
            top2 = __vmaxu2(__vmaxu2(top2, __vmaxu2(finite_magnitudes(x[i].x), finite_magnitudes(x[i].y))),
                            __vmaxu2(finite_magnitudes(x[i].z), finite_magnitudes(x[i].w)));
        top = max(top2 & 0xffffu, top2 >> 16);
    }
    // the group's maximum
#pragma unroll
    for (int o = 1; o < (S::GT < 32 ? S::GT : 32); o <<= 1) top = max(top, __shfl_xor_sync(FULL, top, o));
    if constexpr (S::GT > 32) {
        if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = top;
        __syncthreads();
        top = 0;
#pragma unroll
        for (int w = 0; w < S::GT / 32; ++w) top = max(top, warp_max[group * (S::GT / 32) + w]);
    }
    if (!live) return;

    float scale = fmaxf(e4m3_scale(__half2float(__ushort_as_half((unsigned short)top)), -24), old);
    const float inv = 1.0f / scale;                // exact: powers of two
    const float lim = fminf(448.0f, 61440.0f * inv);
    uint8_t *page_at = (kv ? p.v_pool : p.k_pool) + ((size_t)(p.layer_page0 + blk) * B * H + h) * D;
    // x / scale in fp16 when 1 / scale is one: exact but below 2^-14, far
    // below half of e4m3's smallest, which is stored as 0 either way.
    if (!bad && lim == 448.0f && inv <= 32768.0f) {
        const __half2 by = __float2half2_rn(inv);
#pragma unroll
        for (int i = 0; i < S::VPT; ++i) {
            const int e = i * S::GT + tg;
            const int t = e / CPR, c = e % CPR;
            if (t < lo || t >= hi) continue;
            *reinterpret_cast<uint2 *>(page_at + (size_t)t * H * D + c * 8) =
                make_uint2(scaled_e4m3x2(x[i].x, by) | (scaled_e4m3x2(x[i].y, by) << 16),
                           scaled_e4m3x2(x[i].z, by) | (scaled_e4m3x2(x[i].w, by) << 16));
        }
    } else {
#pragma unroll
        for (int i = 0; i < S::VPT; ++i) {
            const int e = i * S::GT + tg;
            const int t = e / CPR, c = e % CPR;
            if (t < lo || t >= hi) continue;
            float f[8];
            half8_to_float(x[i], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = f[k] != f[k] ? 0.0f : fminf(fmaxf(f[k] * inv, -lim), lim);
            *reinterpret_cast<uint2 *>(page_at + (size_t)t * H * D + c * 8) =
                make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16), e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
        }
    }
    if (lo == 0 || scale > old) {
        if (tg == 0) *scale_at = scale;
        if (lo > 0) {
            // earlier rows, rounded again to the larger scale
            const float ratio = old * inv;
            for (int e = tg; e < lo * CPR; e += S::GT) {
                uint2 *at = reinterpret_cast<uint2 *>(page_at + (size_t)(e / CPR) * H * D + (e % CPR) * 8);
                const uint2 was = *at;
                uint32_t now[2];
                const uint32_t w[2] = {was.x, was.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 a = __half22float2(widen_e4m3(w[k])), b = __half22float2(widen_e4m3(w[k] >> 16));
                    now[k] = e4m3x2(a.x * ratio, a.y * ratio) | (e4m3x2(b.x * ratio, b.y * ratio) << 16);
                }
                *at = make_uint2(now[0], now[1]);
            }
        }
    }
}

template <int B>
int launch_append_b(const AppendArgs &a, AppendParams p, cudaStream_t stream) {
    const int D = a.pool->head_dim;
    const int groups = D == 64 ? AppendShape<B, 64>::GROUPS : AppendShape<B, 128>::GROUPS;
    const long long tasks = (long long)p.max_pages * 2 * p.n_kv_heads;
    const long long per_seq = (tasks + groups - 1) / groups;
    if (per_seq * a.n_seqs > 0x7fffffffll || tasks > 0x7fffffffll)
        return set_error(PF_ERR_INVALID, "pf_append_kv: too many new tokens for one launch");
    p.blocks_per_seq = (int)per_seq;
    const unsigned grid = (unsigned)(per_seq * a.n_seqs);
    if (D == 64) append_kernel<B, 64><<<grid, kThreads, 0, stream>>>(p);
    else append_kernel<B, 128><<<grid, kThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "pf_append_kv: launch");
    return PF_OK;
}

// ----------------------------------------------------------------- gather

constexpr int kGatherRows = 32;

struct GatherParams {
    const uint8_t *k_pool;
    const uint8_t *v_pool;
    const float *k_scale;
    const float *v_scale;
    __half *k_out;
    __half *v_out;
    const int32_t *bt;
    const int32_t *lens;
    const int64_t *cu_off;
    int *status;
    int n_seqs;
    int max_blocks;
    int n_blocks;
    int block_size;
    int n_kv_heads;
    int head_dim;
    long long layer_page0;
};

// CTA (x, y) widens rows x * 32 .. of sequence y, y + gridDim.y, ...; 8 codes
// per thread at a time.  1 byte read and 2 written per value.
__global__ void __launch_bounds__(kThreads) gather_e4m3_kernel(const GatherParams p) {
    const int H = p.n_kv_heads, D = p.head_dim;
    const int vecs = H * D / 8;
    for (int s = blockIdx.y; s < p.n_seqs; s += gridDim.y) {
        int L = p.lens[s];
        const int most = p.max_blocks * p.block_size;
        if (L < 0 || L > most) {
            if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.status, PF_DEV_BAD_LENGTH);
            L = L < 0 ? 0 : most;
        }
        const int64_t row0 = p.cu_off[s];
        for (int r0 = (int)blockIdx.x * kGatherRows; r0 < L; r0 += (int)gridDim.x * kGatherRows) {
            const int n = min(kGatherRows, L - r0) * vecs;
            for (int e = threadIdx.x; e < 2 * n; e += kThreads) {
                const int kv = e >= n, i = kv ? e - n : e;
                const int t = r0 + i / vecs, c = i % vecs;
                const int blk = p.bt[(size_t)s * p.max_blocks + t / p.block_size];
                if (blk < 0 || blk >= p.n_blocks) {
                    atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                    continue;
                }
                const size_t page = (size_t)(p.layer_page0 + blk);
                const uint2 w = *reinterpret_cast<const uint2 *>(
                    (kv ? p.v_pool : p.k_pool) + ((page * p.block_size + t % p.block_size) * vecs + c) * 8);
                const float f = (kv ? p.v_scale : p.k_scale)[page * H + c * 8 / D];
                const uint32_t in[2] = {w.x, w.y};
                uint32_t out[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 a = __half22float2(widen_e4m3(in[k / 2] >> (16 * (k & 1))));
                    const __half2 b = __floats2half2_rn(a.x * f, a.y * f);
                    out[k] = *reinterpret_cast<const uint32_t *>(&b);
                }
                st_stream(reinterpret_cast<uint4 *>((kv ? p.v_out : p.k_out) + ((size_t)(row0 + t) * vecs + c) * 8),
                          make_uint4(out[0], out[1], out[2], out[3]));
            }
        }
    }
}

}  // namespace

int launch_append(const AppendArgs &a, cudaStream_t stream) {
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    const pf_pool *pool = a.pool;
    const int B = pool->block_size;
    AppendParams p;
    p.k_new = static_cast<const __half *>(a.k_new);
    p.v_new = static_cast<const __half *>(a.v_new);
    p.k_pool = static_cast<uint8_t *>(pool->k_base);
    p.v_pool = static_cast<uint8_t *>(pool->v_base);
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.bt = a.block_tables;
    p.lens = a.context_lens;
    p.cu = a.cu_new;
    p.status = status;
    p.max_blocks = a.max_blocks;
    p.max_new = a.max_new;
    p.n_blocks = pool->n_blocks;
    p.n_kv_heads = pool->n_kv_heads;
    // (max_new is a bound that may be loose: no more new tokens than the table holds)
    const long long most_new = std::min((long long)a.max_new, (long long)a.max_blocks * B);
    p.max_pages = (int)((most_new - 1 + B - 1) / B + 1);
    p.layer_page0 = (long long)a.layer * pool->n_blocks;
    switch (B) {
        case 1: return launch_append_b<1>(a, p, stream);
        case 16: return launch_append_b<16>(a, p, stream);
        case 64: return launch_append_b<64>(a, p, stream);
        default: return launch_append_b<256>(a, p, stream);
    }
}

int launch_gather_e4m3(const GatherArgs &a, cudaStream_t stream) {
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    const pf_pool *pool = a.pool;
    GatherParams p;
    p.k_pool = static_cast<const uint8_t *>(pool->k_base);
    p.v_pool = static_cast<const uint8_t *>(pool->v_base);
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    p.k_out = static_cast<__half *>(a.k_out);
    p.v_out = static_cast<__half *>(a.v_out);
    p.bt = a.block_tables;
    p.lens = a.context_lens;
    p.cu_off = a.cu_off;
    p.status = status;
    p.n_seqs = a.n_seqs;
    p.max_blocks = a.max_blocks;
    p.n_blocks = pool->n_blocks;
    p.block_size = pool->block_size;
    p.n_kv_heads = pool->n_kv_heads;
    p.head_dim = pool->head_dim;
    p.layer_page0 = (long long)a.layer * pool->n_blocks;
    const long long blocks = ((long long)a.max_blocks * pool->block_size + kGatherRows - 1) / kGatherRows;
    const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)(a.n_seqs < 65535 ? a.n_seqs : 65535));
    gather_e4m3_kernel<<<grid, kThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "pf_gather_kv: launch");
    return PF_OK;
}

}  // namespace pkv
