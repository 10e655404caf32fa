// norm_rope.cu -- pf_norm_rope_write: RMS norms of queries and keys for each
// head, the position rotation, and the write of K and V into their pages, in
// one pass over a layer's new rows.
//
// For a row x of D values of a q- or k-head, weights w and a token at position p:
//   y   = x * rsqrt(mean(x^2) + eps) * w                        (or y = x)
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i),  c_i = angles[p][i],
//                                              s_i = angles[p][rot / 2 + i],
// over the pairs (y_i, y_{i + rot / 2}), or (y_2i, y_2i+1), i < rot / 2.  All in
// fp32 and rounded once, to the fp16 result.  V rows are copied.
//
// Floor: 2 bytes read and 2 written per value, so it is HBM's.  A row is
// spread over D / 8 lanes, 16 bytes each: the norm is a butterfly among them, the
// partner of a pair (i, i + rot / 2) lies in the lane rot / 16 chunks away and comes
// as the fp16 values read, before the norm (4 shuffles instead of 8).  A group
// of D / 8 lanes takes up to kRows heads of one token, all loads of which are on
// their way before the first is used, and reads the token's cosines and sines
// (fp32, from L2) once for them.
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
        x[r] = r < n ? *reinterpret_cast<const uint4 *>(src + r * D) : make_uint4(0u, 0u, 0u, 0u);

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
        if (dense) *reinterpret_cast<uint4 *>(dense + at) = v;
        if (page) *reinterpret_cast<uint4 *>(page + at) = v;
    };
    if (kind == 2) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (r < n) store(r, x[r]);
        return;
    }

    // the lane's place in the rotation: its pairs, and the chunk of their other halves
    const bool turns = c < p.rot / 8;
    const int half = p.rot / 16;                     // chunks of half the rotated values
    const int partner = INTERLEAVED || !turns ? c : (c < half ? c + half : c - half);
    float cs[8], sn[8];                              // (interleaved: 4 of each)
    if (INTERLEAVED) {
        float both[8] = {1.0f, 1.0f, 1.0f, 1.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (turns) {
            const float *at = p.angles + (size_t)rp * p.rot + c * 4;
            const float4 a = __ldg(reinterpret_cast<const float4 *>(at)), b = __ldg(reinterpret_cast<const float4 *>(at + p.rot / 2));
            both[0] = a.x, both[1] = a.y, both[2] = a.z, both[3] = a.w;
            both[4] = b.x, both[5] = b.y, both[6] = b.z, both[7] = b.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = both[i], sn[i] = both[4 + i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
        if (turns) {
            const float *at = p.angles + (size_t)rp * p.rot + (c < half ? c : c - half) * 8;
            load8(at, cs);
            load8(at + p.rot / 2, sn);
            if (c < half) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
            }
        }
    }
    const float *weight = p.weight[kind];
    float w[8], wp[8];
    if (weight) {
        load8(weight + c * 8, w);
        if (!INTERLEAVED) load8(weight + partner * 8, wp);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (r >= n) break;                           // (the group's lanes together)
        float y[8];
        half8_to_float(x[r], y);
        uint4 xp = x[r];
        if (!INTERLEAVED && p.rot) {
            xp.x = __shfl_sync(group, x[r].x, partner, CPR);
            xp.y = __shfl_sync(group, x[r].y, partner, CPR);
            xp.z = __shfl_sync(group, x[r].z, partner, CPR);
            xp.w = __shfl_sync(group, x[r].w, partner, CPR);
        }
        float yp[8];
        half8_to_float(xp, yp);
        if (weight) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
            for (int o = CPR / 2; o; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
            const float inv = rsqrtf(sum * (1.0f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] *= inv * w[i];
                if (!INTERLEAVED) yp[i] *= inv * wp[i];
            }
        }
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = y[2 * i], b = y[2 * i + 1];
            if (turns) {                             // (the others are not multiplied by a 1 and a 0: infinities stay)
                if (INTERLEAVED) {
                    const float a0 = a;
                    a = fmaf(a0, cs[i], -b * sn[i]);
                    b = fmaf(b, cs[i], a0 * sn[i]);
                } else {
                    a = fmaf(a, cs[2 * i], yp[2 * i] * sn[2 * i]);
                    b = fmaf(b, cs[2 * i + 1], yp[2 * i + 1] * sn[2 * i + 1]);
                }
            }
            const __half2 h = __floats2half2_rn(a, b);
            out[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        store(r, make_uint4(out[0], out[1], out[2], out[3]));
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
