// norm_rope.cu -- pf_norm_rope_write: RMS norms of queries and keys for each
// head, the position rotation, and the write of K and V into their pages, in
// one pass over a layer's new rows.
//
// For a row x of D values of a q- or k-head, weights w and a token at position p:
//   y   = x * rsqrt(mean(x^2) + eps) * w                        (or y = x)
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i),  c_i = angles[p][i],
//                                              s_i = angles[p][rot / 2 + i],
// over the pairs (y_i, y_{i + rot / 2}), or (y_2i, y_2i+1), i < rot / 2.  All in
// fp32 and rounded once, to the fp16 result.  V rows are copied, and so are chunks
// without a norm outside the rotated part.
//
// Floor: 2 bytes read and 2 written per value, so it is HBM's.  Measured on
// GB300: four prompts of 2,048 tokens, 40 heads x 128 (503 MB) 87 us, 5.8 TB/s,
// 85 % of the measured copy rate; one token each for 4 and 256 sequences 3 to
// 3.6 us, a launch and a chain of dependent loads.  A row is spread over D / 8
// lanes, 16 bytes each: the norm is a butterfly among them, the partner of a pair
// (i, i + rot / 2) lies in the lane rot / 16 chunks away and comes as the fp16
// values read, before the norm.  A group of D / 8 lanes takes up to kRows heads of
// one token, all loads of which are on their way before the first is used, and
// folds the token's cosines and sines (fp32, from L2) and the weights into two
// factors per value, once for them.  Instructions count: with the norm, weights
// and rotation one after another the prompts took 106 us; with the two factors and
// two-wide fp32 instructions 92; with streaming stores 87.  (kRows 2, 4, 8 at 128
// threads: 111, 87, 88 us, the 4 sequences 3.0, 3.6, 4.5; 256 threads a CTA were
// slower, 108 us with 4, its CTAs ending less evenly.)
#include <algorithm>

#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 4;   // heads of a token per group of lanes

struct RopeParams {
    const __half *x[3];        // q, k, v rows
    long long stride[3];       // values between tokens
    __half *q_out;
    __half *k_out;             // null: not wanted
    long long q_out_stride;
    long long k_out_stride;
    const float *weight[2];    // of q, of k; null: no norm
    const float *angles;
    const int32_t *rope_pos;   // null: pos
    __half *k_pool;            // null: no cache write
    __half *v_pool;
    const int32_t *bt;
    const int32_t *seq_idx;
    const int32_t *pos;
    int *status;
    float eps;
    int n_positions;
    int rot;
    int n_q_heads;
    int n_kv_heads;
    int q_items;               // groups per token: of q, of k (and as many of v)
    int k_items;
    int items;                 // of a token
    unsigned n_items;
    int n_table_rows;
    int max_blocks;
    int n_blocks;
    int block_size;
    long long layer_row0;
};

// 16 bytes read once (coherent: outputs may be the inputs, in place).
__device__ __forceinline__ uint4 ld_once(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Pairs of fp32 values for the two-wide instructions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t widen(uint32_t half2_bits) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&half2_bits));
    return pair(f.x, f.y);
}
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
    const float2 f = both(v);
    return pair(f.y, f.x);
}
// Eight floats.
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeParams p) {
    constexpr int CPR = D / 8;                       // lanes (16-byte chunks) of a row
    const unsigned item = blockIdx.x * (unsigned)(kThreads / CPR) + threadIdx.x / CPR;
    if (item >= p.n_items) return;                   // whole groups: shuffles stay within one
    const int c = (int)threadIdx.x % CPR;
    const int lane = (int)threadIdx.x % 32;
    const unsigned group = (CPR == 32 ? 0xffffffffu : ((1u << CPR) - 1u)) << (lane & ~(CPR - 1));
    const int token = (int)(item / (unsigned)p.items);
    int sub = (int)(item - (unsigned)token * (unsigned)p.items);
    // what this group takes: heads h0 .. h0 + n - 1 of q (0), k (1) or v (2)
    int kind = 0, heads = p.n_q_heads;
    if (sub >= p.q_items) {
        sub -= p.q_items;
        heads = p.n_kv_heads;
        kind = 1;
        if (sub >= p.k_items) {
            sub -= p.k_items;
            kind = 2;
        }
    }
    const int h0 = sub * kRows;
    const int n = min(kRows, heads - h0);
    const __half *src = p.x[kind] + (long long)token * p.stride[kind] + h0 * D + c * 8;
    uint4 x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        x[r] = r < n ? ld_once(reinterpret_cast<const uint4 *>(src + r * D)) : make_uint4(0u, 0u, 0u, 0u);

    // the token's angles, and its slot
    const bool rotated = p.rot && kind < 2;
    const int rp = !rotated ? 0 : (p.rope_pos ? p.rope_pos[token] : p.pos[token]);
    if (rotated && (rp < 0 || rp >= p.n_positions)) {
        if (c == 0) atomicOr(p.status, PF_DEV_BAD_POSITION);
        return;
    }
    __half *page = nullptr;                          // the token's rows in the pool of this kind
    if (kind && p.k_pool) {
        const int s = p.seq_idx[token], t = p.pos[token];
        if (s < 0 || s >= p.n_table_rows || t < 0 || t / p.block_size >= p.max_blocks) {
            if (c == 0) atomicOr(p.status, PF_DEV_BAD_POSITION);
        } else {
            const int blk = p.bt[(size_t)s * p.max_blocks + t / p.block_size];
            if (blk < 0 || blk >= p.n_blocks) {
                if (c == 0) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
            } else {
                const size_t row = (size_t)(p.layer_row0 + (long long)blk * p.block_size + t % p.block_size);
                page = (kind == 1 ? p.k_pool : p.v_pool) + row * (size_t)p.n_kv_heads * D;
            }
        }
    }
    __half *dense = nullptr;
    if (kind == 0) dense = p.q_out + (long long)token * p.q_out_stride;
    if (kind == 1 && p.k_out) dense = p.k_out + (long long)token * p.k_out_stride;
    auto store = [&](int r, uint4 v) {
        const int at = (h0 + r) * D + c * 8;
        if (dense) st_stream(reinterpret_cast<uint4 *>(dense + at), v);
        if (page) st_stream(reinterpret_cast<uint4 *>(page + at), v);
    };
    if (kind == 2) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (r < n) store(r, x[r]);
        return;
    }

    // The lane's eight values x and their partners p (the other values of their
    // pairs) become inv * (x A + p B), A = w c and B = -+ w' s with the partner's
    // weight w': the token's, for all of its rows.
    const bool turns = c < p.rot / 8;
    const int half = p.rot / 16;                     // chunks of half the rotated values
    const int partner = INTERLEAVED || !turns ? c : (c < half ? c + half : c - half);
    const float *weight = p.weight[kind];
    float w[8], wp[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = wp[i] = 1.0f;
    if (weight) {
        load8(weight + c * 8, w);
        if (!INTERLEAVED) load8(weight + partner * 8, wp);
    }
    uint64_t A[4], B[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        A[i] = pair(w[2 * i], w[2 * i + 1]);
        B[i] = 0;
    }
    if (turns) {
        const float *at = p.angles + (size_t)rp * p.rot;
        if (INTERLEAVED) {
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(at + c * 4)),
                         s4 = __ldg(reinterpret_cast<const float4 *>(at + p.rot / 2 + c * 4));
            const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                A[i] = mul2(A[i], pair(cs[i], cs[i]));
                B[i] = mul2(pair(w[2 * i + 1], w[2 * i]), pair(-sn[i], sn[i]));
            }
        } else {
            float cs[8], sn[8];
            const int j = (c < half ? c : c - half) * 8;
            load8(at + j, cs);
            load8(at + p.rot / 2 + j, sn);
            const float sign = c < half ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                A[i] = mul2(A[i], pair(cs[2 * i], cs[2 * i + 1]));
                B[i] = mul2(pair(sign * wp[2 * i], sign * wp[2 * i + 1]), pair(sn[2 * i], sn[2 * i + 1]));
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (r >= n) break;                           // (the group's lanes together)
        const uint32_t in[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
        uint64_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = widen(in[i]);
        uint64_t inv = 0;
        if (weight) {
            uint64_t sum2 = mul2(y[0], y[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) sum2 = fma2(y[i], y[i], sum2);
            const float2 s2 = both(sum2);
            float sum = s2.x + s2.y;
#pragma unroll
            for (int o = CPR / 2; o; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
            const float f = rsqrtf(sum * (1.0f / D) + p.eps);
            inv = pair(f, f);
        }
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t v = mul2(y[i], A[i]);
            if (p.rot) {
                // (lanes that do not turn take and add nothing: infinities stay
                // their rows', zeros keep their signs)
                if (INTERLEAVED) {
                    if (turns) v = fma2(swapped(y[i]), B[i], v);
                } else {
                    const uint32_t bits = __shfl_sync(group, in[i], partner, CPR);
                    if (turns) v = fma2(widen(bits), B[i], v);
                }
            }
            if (weight) v = mul2(v, inv);
            const float2 o = both(v);
            const __half2 h = __floats2half2_rn(o.x, o.y);
            out[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        // neither normed nor turned: as they are, NaNs too
        store(r, weight || turns ? make_uint4(out[0], out[1], out[2], out[3]) : x[r]);
    }
}

}  // namespace

int launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream) {
    int *status = device_status_ptr();
    if (!status) return PF_ERR_CUDA;
    const pf_pool *pool = a.pool;
    const int D = pool->head_dim;
    const bool cached = a.block_tables != nullptr;
    RopeParams p;
    const void *x[3] = {a.q, a.k, a.v};
    const long long strides[3] = {a.q_stride, a.k_stride, a.v_stride};
    for (int i = 0; i < 3; ++i) {
        p.x[i] = static_cast<const __half *>(x[i]);
        p.stride[i] = strides[i];
    }
    p.q_out = static_cast<__half *>(a.q_out);
    p.k_out = static_cast<__half *>(a.k_out);
    p.q_out_stride = a.q_out_stride;
    p.k_out_stride = a.k_out_stride;
    p.weight[0] = a.q_weight;
    p.weight[1] = a.k_weight;
    p.angles = a.angles;
    p.rope_pos = a.rope_pos;
    p.k_pool = cached ? static_cast<__half *>(pool->k_base) : nullptr;
    p.v_pool = cached ? static_cast<__half *>(pool->v_base) : nullptr;
    p.bt = a.block_tables;
    p.seq_idx = a.seq_idx;
    p.pos = a.pos;
    p.status = status;
    p.eps = a.eps;
    p.n_positions = a.n_positions;
    p.rot = a.rot_dim;
    p.n_q_heads = a.n_q_heads;
    p.n_kv_heads = pool->n_kv_heads;
    p.q_items = (a.n_q_heads + kRows - 1) / kRows;
    p.k_items = a.k ? (pool->n_kv_heads + kRows - 1) / kRows : 0;
    p.items = p.q_items + p.k_items * (cached ? 2 : 1);
    p.n_table_rows = a.n_table_rows;
    p.max_blocks = a.max_blocks;
    p.n_blocks = pool->n_blocks;
    p.block_size = pool->block_size;
    p.layer_row0 = (long long)a.layer * pool->n_blocks * pool->block_size;
    // a launch counts its groups in 31 bits: more tokens are consecutive launches
    const int per_launch = (int)std::min<long long>(a.n_tokens, 0x7fffffffll / p.items);
    for (long long t0 = 0; t0 < a.n_tokens; t0 += per_launch) {
        RopeParams l = p;
        const int n = (int)std::min<long long>(per_launch, a.n_tokens - t0);
        for (int i = 0; i < 3; ++i)
            if (l.x[i]) l.x[i] += t0 * l.stride[i];
        if (l.q_out) l.q_out += t0 * l.q_out_stride;
        if (l.k_out) l.k_out += t0 * l.k_out_stride;
        if (l.rope_pos) l.rope_pos += t0;
        if (l.seq_idx) l.seq_idx += t0;
        if (l.pos) l.pos += t0;
        l.n_items = (unsigned)n * (unsigned)p.items;
        const unsigned groups = (unsigned)(kThreads / (D / 8));
        const unsigned grid = (l.n_items + groups - 1) / groups;
        if (D == 64) {
            if (a.interleaved) norm_rope_kernel<64, true><<<grid, kThreads, 0, stream>>>(l);
            else norm_rope_kernel<64, false><<<grid, kThreads, 0, stream>>>(l);
        } else {
            if (a.interleaved) norm_rope_kernel<128, true><<<grid, kThreads, 0, stream>>>(l);
            else norm_rope_kernel<128, false><<<grid, kThreads, 0, stream>>>(l);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_error(e, "pf_norm_rope_write: launch");
    }
    return PF_OK;
}

}  // namespace pkv
