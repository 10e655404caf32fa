// rows_attention.cuh -- attention of a few query rows per (sequence, kv-head)
// over the paged cache: decode and short appends over an e4m3 pool, short
// cross attention over either pool type.
//
// For a (sequence s, kv-head h) with L tokens and at most 16 query rows (its
// query tokens x its gh q-heads, row r = i * gh + g of token i):
//   z_rt = scale * q_r . K_t,  out_r = sum_t softmax_t(z_r) V_t,
// t < L (cross, decode) or t <= L - n + i (causal).  e4m3 pools: K_t = code *
// k_scale[page][h], V_t = code * v_scale[page][h].
//
// Bound: every K and V byte of the context is read once and used for at most
// 16 rows, so HBM bounds it; the rest is kept below that.
// * Work: stages of ST tokens (a 4 KB piece of K and V for one head at 64-
//   and 128-byte rows).  The stages of all (sequence, group of HG kv-heads)
//   pairs are cut into equal spans, one per team of HG warps; warp hl of a
//   team walks the span for head hl, so the warps of a team read neighbouring
//   runs of the same page rows at about the same time.  There is no barrier
//   between warps.
// * Each warp runs its own ring of NST stages filled by 16-byte cp.async (4
//   bytes for the scales) and never leaves a stage to another warp, so
//   wait_group and __syncwarp are all the synchronisation.  Rows past L and
//   rows of bad pages are zero-filled, so nothing unwritten is read.
// * Products on warp-level MMA m16n8k16 with the tokens on the M side and the
//   rows on the N side: S^T = K Q^T and O^T = V^T P^T.  With at most 8 rows
//   that is half the MMAs of the other order.  The k order of the first
//   product and the row and column orders of the second are free, so each
//   lane reads 16-byte chunks of K rows as they lie, and a run of D / 8
//   neighbouring dims of four V rows; e4m3 pairs of two tokens are
//   interleaved by byte permutes before they are widened to fp16 (exact).
// * Softmax in the log2 domain on the S^T fragments, fp32.  The running
//   maximum is raised only when a lane sees a score 2^8 above it, so its
//   reduction over the lanes is off the common path; the row sums stay per
//   lane until the end.
// * The K scale multiplies the score, the V scale the weight before it is
//   rounded to fp16 for the second product.  Weights are held relative to the
//   largest V scale met so far (v_ref), shifted up by 2^7: at most 2^15, and
//   the smallest normal fp16 weight is 2^-21 of the largest scale's.  The row
//   sum is the fp32 weights' own.  fp32 output takes the product twice, with
//   the weight's fp16 part and with its rounding error.
// * A pair cut between spans leaves its parts (acc, m, l) in the workspace;
//   the warp that finds itself the last of the pair's parts (a counter per
//   cut, stamped with the launch's epoch and cleared by that warp) merges
//   them with the log-sum-exp rule.  Nobody waits for anybody.
#pragma once

#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace rows {

constexpr int NW = 12;               // warps per CTA: teams of 1, 2, 3 or 4
constexpr int NTHREADS = 32 * NW;
constexpr int kMaxSeqs = 1024;       // sequences per launch
constexpr float kRaiseLog2 = 8.0f;   // raise the running maximum past 2^8
constexpr float kNoScore = -1.0e30f; // the running maximum before any score
constexpr float kWeightShift = 128.0f;
constexpr unsigned FULL = 0xffffffffu;

// Cost of a (sequence, group) pair in the partition, in stages: entering one
// costs a q load, a merge of lanes and a store.
constexpr int kPairCost = 1;

struct Params {
    const __half *q;
    const uint8_t *k_pool;
    const uint8_t *v_pool;
    const float *k_scale;   // e4m3 pools, else null
    const float *v_scale;
    void *out;
    const int32_t *bt;
    const int32_t *lens;
    const int32_t *cu_q;    // null: one query token per sequence, row s
    int *status;
    unsigned long long *counters;   // one per (team, head): arrivals of the pair that the team cuts last
    float *recs;                    // [team][2][head][rows][D + 4]: parts of cut pairs
    unsigned epoch;
    int n_seqs;
    int max_blocks;
    int n_blocks;
    int block_size;
    int block_shift;        // log2 of block_size
    int n_q_heads;
    int n_kv_heads;
    int gh;
    int hg;                 // kv-heads (warps) per team
    int n_groups;
    int rows;               // rows per kv-head the call allows
    int causal;
    int out_f32;
    long long layer_row0;   // layer * n_blocks * block_size
    long long layer_page0;  // layer * n_blocks
    float scale_log2;
};

template <typename T, int D>
struct Shape {
    static constexpr bool Q8 = sizeof(T) == 1;
    static constexpr int RB = D * (int)sizeof(T);    // bytes of one head's row
    static constexpr int U = RB == 64 ? 2 : 1;       // 16-token tiles per stage
    static constexpr int ST = 16 * U;                // tokens per stage
    static constexpr int KV = ST * RB;               // K (or V) bytes of a stage
    static constexpr int STAGE = 2 * KV + (Q8 ? ST * 8 : 0);
    static constexpr int NST = RB == 256 ? 2 : 4;
    static constexpr int SMEM = NW * NST * STAGE;
    static constexpr int NRUN = RB == 256 ? 2 : 1;   // runs of neighbouring dims a lane holds of O
    static constexpr int RL = D / 8 / NRUN;          // dims per run
};

// Work units in order (sequence, group, stage): a pair has kPairCost units
// without work, then its stages.  W units are cut into n = min(W, teams)
// spans; team j takes [start(j), start(j + 1)).
struct Spans {
    long long W, n;
    __device__ __forceinline__ long long start(long long j) const { return j >= n ? W : W * j / n; }
    __device__ __forceinline__ long long owner(long long x) const { return ((x + 1) * n - 1) / W; }
};

// Walks the stages of one team's span.
struct Cursor {
    int s;             // sequence; n_seqs: done
    int g;             // group
    int tile;          // next stage of the pair
    int end;           // one past the span's last stage of the pair
    int n_tiles;       // stages of the pair
};

__device__ __forceinline__ uint32_t cvt2_e4m3(uint32_t pair) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(pair));
    return h;
}
__device__ __forceinline__ uint32_t cvt2_e4m3_hi(uint32_t pair) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(pair));
    return h;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_f16_16816(d, a, b0, b1);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Copies that read `bytes` bytes (all or none) and zero-fill the rest.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}

// Token p of a 16-token tile sits in row `slot` of the MMA's M side: lane t
// of a quad then needs V rows t, t + 4, t + 8, t + 12, which the V layout
// below reads without bank conflicts.
__device__ __forceinline__ int slot_of(int p) { return (p & 8) + 2 * (p & 3) + ((p >> 2) & 1); }
__device__ __forceinline__ int token_of(int slot) { return (slot & 8) + ((slot >> 1) & 3) + 4 * (slot & 1); }

// Shared-memory offset of 16-byte chunk c of K slot r / V token r in a tile.
template <int RB>
__device__ __forceinline__ uint32_t k_off(int r, int c) {
    return (uint32_t)(r * RB + ((RB == 64 ? c : c ^ ((r & 1) << 2)) << 4));
}
template <int RB>
__device__ __forceinline__ uint32_t v_off(int r, int c) {
    return (uint32_t)(r * RB + ((RB == 64 ? c ^ (r & 2) : c ^ ((r & 3) << 1)) << 4));
}

// Clamped context length of sequence s; flags what the call does not allow.
// A sequence without query tokens has no work.
__device__ __forceinline__ int context_length(const Params &p, int s, bool flag) {
    int L = p.lens[s];
    const long long most = (long long)p.max_blocks * p.block_size;
    int bad = 0;
    if (L < 0 || L > most) {
        bad = 1;
        L = L < 0 ? 0 : (int)most;
    }
    if (p.cu_q) {
        const int n = p.cu_q[s + 1] - p.cu_q[s];
        if (n < 0 || (long long)n * p.gh > p.rows || (p.causal && n > L)) bad = 1;
        if (n <= 0) L = 0;
    }
    if (bad && flag) atomicOr(p.status, PF_DEV_BAD_LENGTH);
    return L;
}

template <typename T, int D, int NT, bool HILO>
__global__ void __launch_bounds__(NTHREADS, 1) rows_attention_kernel(const Params p) {
    using S = Shape<T, D>;
    constexpr int RB = S::RB;
    constexpr int U = S::U;
    constexpr int ST = S::ST;
    constexpr int CPR = RB / 16;         // 16-byte chunks of a row
    constexpr int KS = D / 16;           // k-steps of the scores
    constexpr int MT = D / 16;           // 16-dim tiles of O
    constexpr int REC = D + 4;           // floats of a row's record
    constexpr bool Q8 = S::Q8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long pre[kMaxSeqs + 1];   // units before sequence s
    __shared__ int len_sh[kMaxSeqs];
    __shared__ long long warp_sum[NW];

    const int warp = (int)threadIdx.x / 32;
    const int lane = (int)threadIdx.x % 32;

    // Prefix of the units over the sequences: each thread scans a run of
    // consecutive ones.
    {
        const int per = (p.n_seqs + NTHREADS - 1) / NTHREADS;
        const int s0 = min((int)threadIdx.x * per, p.n_seqs);
        const int s1 = min(s0 + per, p.n_seqs);
        long long mine = 0;
        for (int s = s0; s < s1; ++s) {
            const int L = context_length(p, s, blockIdx.x == 0);
            len_sh[s] = L;
            if (L > 0) mine += (long long)((L + ST - 1) / ST + kPairCost) * p.n_groups;
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        long long base = 0;
        for (int w = 0; w < warp; ++w) base += warp_sum[w];
        long long at = base + incl - mine;
        for (int s = s0; s < s1; ++s) {
            pre[s] = at;
            const int L = len_sh[s];
            if (L > 0) at += (long long)((L + ST - 1) / ST + kPairCost) * p.n_groups;
        }
        if (threadIdx.x == NTHREADS - 1) pre[p.n_seqs] = at;
        __syncthreads();
    }

    // Rows of empty contexts: zeros.
    for (int s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
        if (p.lens[s] > 0) continue;
        const int r0 = p.cu_q ? p.cu_q[s] : s;
        const int n = p.cu_q ? min(p.cu_q[s + 1] - r0, p.rows / p.gh) : 1;
        const size_t row = (size_t)p.n_q_heads * D;
        for (size_t e = threadIdx.x; n > 0 && e < (size_t)n * row / 8; e += NTHREADS) {
            if (p.out_f32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + r0 * row) + 2 * e;
                o[0] = o[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            } else {
                reinterpret_cast<uint4 *>(static_cast<__half *>(p.out) + r0 * row)[e] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }

    const int hl = warp % p.hg;
    const int teams_per_cta = NW / p.hg;
    const long long teams = (long long)gridDim.x * teams_per_cta;
    const long long W = pre[p.n_seqs];
    if (warp / p.hg >= teams_per_cta || W == 0) return;
    const long long team = (long long)blockIdx.x * teams_per_cta + warp / p.hg;
    const Spans sp{W, W < teams ? W : teams};
    if (team >= sp.n) return;
    const long long u_lo = sp.start(team), u_hi = sp.start(team + 1);

    // Enter pair (c.s, c.g), or the next one of the span with a stage in it.
    auto settle = [&](Cursor &c) {
        for (;;) {
            while (c.s < p.n_seqs && len_sh[c.s] == 0) {
                ++c.s;
                c.g = 0;
            }
            if (c.s >= p.n_seqs) return;
            c.n_tiles = (len_sh[c.s] + ST - 1) / ST;
            const long long ub = pre[c.s] + (long long)c.g * (c.n_tiles + kPairCost) + kPairCost;   // its first stage
            if (ub >= u_hi) {
                c.s = p.n_seqs;
                return;
            }
            c.tile = (int)max(0ll, u_lo - ub);
            c.end = (int)min((long long)c.n_tiles, u_hi - ub);
            if (c.tile < c.end) return;
            if (++c.g == p.n_groups) {
                c.g = 0;
                ++c.s;
            }
        }
    };
    auto advance = [&](Cursor &c) {
        if (++c.tile < c.end) return;
        if (++c.g == p.n_groups) {
            c.g = 0;
            ++c.s;
        }
        settle(c);
    };

    Cursor look;
    {
        int lo = 0, hi = p.n_seqs - 1;   // the last sequence with pre <= u_lo
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= u_lo) lo = mid;
            else hi = mid - 1;
        }
        look.s = lo;
        look.g = 0;
        if (len_sh[lo] > 0) {
            const long long per = (pre[lo + 1] - pre[lo]) / p.n_groups;
            look.g = (int)((u_lo - pre[lo]) / per);
        }
        settle(look);
    }
    Cursor cur = look;

    // --------------------------------------------------------------- copies
    uint8_t *ring = smem + (size_t)warp * S::NST * S::STAGE;
    const uint32_t ring_s = smem_addr(ring);
    const size_t tok_bytes = (size_t)p.n_kv_heads * RB;
    constexpr int PF = S::NST - 1;       // stages in flight, and block ids looked up ahead
    // the next PF stages to copy: this lane's token (lane mod ST) of each
    int f_id[PF], f_off[PF], f_h[PF];    // block id (-2: no token), row in the page, kv-head
    auto look_up = [&](int &id, int &off, int &h) {
        id = -2;
        off = 0;
        h = -1;                          // nothing to copy
        if (look.s >= p.n_seqs) return;
        const int t = look.tile * ST + (lane & (ST - 1));
        h = look.g * p.hg + hl;
        if (h >= p.n_kv_heads) h = -1;   // no such head in the last group
        else if (t < len_sh[look.s]) {
            id = p.bt[(size_t)look.s * p.max_blocks + (t >> p.block_shift)];
            off = t & (p.block_size - 1);
        }
        advance(look);
    };
    auto copy = [&](int stage, int id, int off, int h) {
        const uint32_t base = ring_s + stage * S::STAGE;
        if (h >= 0) {
            long long row = -1;
            int page = -1;
            if (id >= 0 && id < p.n_blocks) {
                row = p.layer_row0 + (long long)id * p.block_size + off;
                page = id;
            } else if (id != -2) {
                atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
            }
            const int row32 = (int)row;  // below 2^31: checked when the pool was made
#pragma unroll
            for (int i = 0; i < ST * CPR / 32; ++i) {
                const int e = i * 32 + lane;
                const int tok = e / CPR, c = e % CPR;
                const int r = __shfl_sync(FULL, row32, tok);
                const size_t at = r < 0 ? 0 : (size_t)r * tok_bytes + (size_t)h * RB + c * 16;
                const uint32_t n = r < 0 ? 0u : 16u;
                const int u = tok / 16, pt = tok % 16;
                cp16(base + u * 16 * RB + k_off<RB>(slot_of(pt), c), p.k_pool + at, n);
                cp16(base + S::KV + u * 16 * RB + v_off<RB>(pt, c), p.v_pool + at, n);
            }
            if constexpr (Q8) {
                const size_t at = page < 0 ? 0 : (size_t)(p.layer_page0 + page) * p.n_kv_heads + h;
                const uint32_t n = page < 0 ? 0u : 4u;
                const uint32_t sc = base + 2 * S::KV;
                if constexpr (ST == 32) {
                    cp4(sc + lane * 4, p.k_scale + at, n);
                    cp4(sc + ST * 4 + lane * 4, p.v_scale + at, n);
                } else {
                    cp4(sc + lane * 4, (lane < ST ? p.k_scale : p.v_scale) + at, n);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < PF; ++k) look_up(f_id[k], f_off[k], f_h[k]);
#pragma unroll
    for (int k = 0; k < PF; ++k) {
        copy(k, f_id[k], f_off[k], f_h[k]);
        look_up(f_id[k], f_off[k], f_h[k]);
    }

    // ----------------------------------------------------------------- math
    const int gq = lane >> 2;            // N row of a B fragment, M row of an A fragment
    const int tq = lane & 3;
    int stage = 0;
    while (cur.s < p.n_seqs) {
        const int s = cur.s;
        const int h = cur.g * p.hg + hl;
        const bool active = h < p.n_kv_heads;
        const int L = len_sh[s];
        const int first = cur.tile, last = cur.end, n_tiles = cur.n_tiles;
        const long long ub = pre[s] + (long long)cur.g * (n_tiles + kPairCost) + kPairCost;
        const int q0 = p.cu_q ? p.cu_q[s] : s;
        const int nq = p.cu_q ? min(p.cu_q[s + 1] - q0, p.rows / p.gh) : 1;
        const int n_rows = nq * p.gh;

        // q as B fragments: lane (gq, tq) of k-step j holds four dims of row
        // gq in the order in which it reads K.
        uint32_t qb[KS][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + gq;
            const bool ok = active && r < n_rows;
            const int i = ok ? r / p.gh : 0;
            const __half *src = p.q + ((size_t)(q0 + i) * p.n_q_heads + (size_t)(active ? h : 0) * p.gh + (ok ? r - i * p.gh : 0)) * D;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const int d = Q8 ? (tq + 4 * (j / 4)) * 16 + (j % 4) * 4 : (tq + 4 * (j / 2)) * 8 + (j % 2) * 4;
                const uint2 x = ok ? *reinterpret_cast<const uint2 *>(src + d) : make_uint2(0u, 0u);
                qb[j][nt][0] = x.x;
                qb[j][nt][1] = x.y;
            }
        }
        int vis[NT][2];                  // tokens that rows 2 tq, 2 tq + 1 see
        int vis_min = L;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * tq + e;
                vis[nt][e] = p.causal && r < n_rows ? max(0, L - nq + r / p.gh + 1) : L;
            }
        }
        if (p.causal) vis_min = max(0, L - nq + 1);

        float m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kNoScore;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int b = 0; b < MT; ++b) o[b][nt][0] = o[b][nt][1] = o[b][nt][2] = o[b][nt][3] = 0.0f;
        }
        float v_ref = 0.0f, v_inv = 0.0f;

        for (int tile = first; tile < last; ++tile) {
            __syncwarp();                // the stage about to be filled has been read by every lane
            {
                const int fill = stage == 0 ? S::NST - 1 : stage - 1;
                copy(fill, f_id[0], f_off[0], f_h[0]);
#pragma unroll
                for (int k = 0; k + 1 < PF; ++k) {
                    f_id[k] = f_id[k + 1];
                    f_off[k] = f_off[k + 1];
                    f_h[k] = f_h[k + 1];
                }
                look_up(f_id[PF - 1], f_off[PF - 1], f_h[PF - 1]);
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(PF) : "memory");
            __syncwarp();
            const uint32_t kb = ring_s + stage * S::STAGE;
            const uint32_t vb = kb + S::KV;
            const uint32_t scb = kb + 2 * S::KV;
            stage = stage + 1 == S::NST ? 0 : stage + 1;
            if (!active) continue;

            // scores of slots gq and gq + 8 for rows 2 tq, 2 tq + 1
            float z[U][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) z[u][nt][0] = z[u][nt][1] = z[u][nt][2] = z[u][nt][3] = 0.0f;
#pragma unroll
                for (int i = 0; i < CPR / 4; ++i) {
                    const uint4 ka = lds128(kb + u * 16 * RB + k_off<RB>(gq, tq + 4 * i));
                    const uint4 kc = lds128(kb + u * 16 * RB + k_off<RB>(gq + 8, tq + 4 * i));
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w};
                    const uint32_t wc[4] = {kc.x, kc.y, kc.z, kc.w};
                    if constexpr (Q8) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t a[4] = {cvt2_e4m3(wa[w]), cvt2_e4m3(wc[w]), cvt2_e4m3_hi(wa[w]),
                                                   cvt2_e4m3_hi(wc[w])};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma(z[u][nt], a, qb[i * 4 + w][nt][0], qb[i * 4 + w][nt][1]);
                        }
                    } else {
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const uint32_t a[4] = {wa[2 * w], wc[2 * w], wa[2 * w + 1], wc[2 * w + 1]};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma(z[u][nt], a, qb[i * 2 + w][nt][0], qb[i * 2 + w][nt][1]);
                        }
                    }
                }
            }
            const int tok0 = tile * ST;
            const bool masked = tok0 + ST > vis_min;
            const int tslot = token_of(gq);
            float vr[U][2];              // weight factors of slots gq, gq + 8
            if constexpr (Q8) {
                float vm = 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        vr[u][e] = lds32(scb + (ST + u * 16 + e * 8 + tslot) * 4);
                        vm = fmaxf(vm, vr[u][e]);
                    }
                }
                vm = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(vm)));   // scales are not negative
                if (vm > v_ref) {
                    const float f = v_ref / vm;
                    v_ref = vm;
                    v_inv = kWeightShift / vm;
#pragma unroll
                    for (int b = 0; b < MT; ++b)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[b][nt][e] *= f;
                }
            }
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float f = p.scale_log2;
                    if constexpr (Q8) f *= lds32(scb + (u * 16 + e * 8 + tslot) * 4);
                    const int t = tok0 + u * 16 + e * 8 + tslot;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float v = z[u][nt][2 * e + x] * f;
                            if (masked && t >= vis[nt][x]) v = -INFINITY;
                            z[u][nt][2 * e + x] = v;
                            mx[nt][x] = fmaxf(mx[nt][x], v);
                        }
                    }
                }
            }
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) raise |= mx[nt][0] > m[nt][0] + kRaiseLog2 || mx[nt][1] > m[nt][1] + kRaiseLog2;
            if (__any_sync(FULL, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v = mx[nt][x];
                        v = fmaxf(v, __shfl_xor_sync(FULL, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(FULL, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(FULL, v, 16));
                        if (v > m[nt][x] + kRaiseLog2) {
                            const float f = ex2(m[nt][x] - v);
                            m[nt][x] = v;
                            l[nt][x] *= f;
#pragma unroll
                            for (int b = 0; b < MT; ++b) {
                                o[b][nt][x] *= f;
                                o[b][nt][2 + x] *= f;
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // weights, transposed into B fragments (tokens x rows)
                uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float w0 = ex2(z[u][nt][2 * e] - m[nt][0]);
                        float w1 = ex2(z[u][nt][2 * e + 1] - m[nt][1]);
                        l[nt][0] += w0;
                        l[nt][1] += w1;
                        if constexpr (Q8) {
                            w0 *= vr[u][e] * v_inv;
                            w1 *= vr[u][e] * v_inv;
                        }
                        const uint32_t hi = pack2(w0, w1);
                        pb[nt][e] = transpose8x8(hi);
                        if constexpr (HILO) {
                            const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                            pl[nt][e] = transpose8x8(pack2(w0 - hf.x, w1 - hf.y));
                        }
                    }
                }
                // O^T += V^T P^T: V rows tq + {0, 4, 8, 12}
#pragma unroll
                for (int run = 0; run < S::NRUN; ++run) {
                    constexpr int WORDS = RB / 32 / S::NRUN;   // 4-byte words of a run
                    uint32_t x[4][WORDS];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = tq + 4 * i;
                        if constexpr (WORDS == 2) {
                            const uint2 v = lds64(vb + u * 16 * RB + v_off<RB>(r, gq >> 1) + (gq & 1) * 8);
                            x[i][0] = v.x;
                            x[i][1] = v.y;
                        } else {
                            const uint4 v = lds128(vb + u * 16 * RB + v_off<RB>(r, gq + 8 * run));
                            x[i][0] = v.x;
                            x[i][1] = v.y;
                            x[i][2] = v.z;
                            x[i][3] = v.w;
                        }
                    }
                    constexpr int TW = Q8 ? 2 : 1;             // 16-dim tiles per word
#pragma unroll
                    for (int w = 0; w < WORDS; ++w) {
#pragma unroll
                        for (int k = 0; k < TW; ++k) {
                            uint32_t a[4];
                            if constexpr (Q8) {
                                const uint32_t sel = k ? 0x7362u : 0x5140u;
                                const uint32_t ab = __byte_perm(x[0][w], x[1][w], sel);
                                const uint32_t cd = __byte_perm(x[2][w], x[3][w], sel);
                                a[0] = cvt2_e4m3(ab);
                                a[1] = cvt2_e4m3_hi(ab);
                                a[2] = cvt2_e4m3(cd);
                                a[3] = cvt2_e4m3_hi(cd);
                            } else {
                                a[0] = __byte_perm(x[0][w], x[1][w], 0x5410);
                                a[1] = __byte_perm(x[0][w], x[1][w], 0x7632);
                                a[2] = __byte_perm(x[2][w], x[3][w], 0x5410);
                                a[3] = __byte_perm(x[2][w], x[3][w], 0x7632);
                            }
                            const int b = (run * WORDS + w) * TW + k;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma(o[b][nt], a, pb[nt][0], pb[nt][1]);
                                if constexpr (HILO) mma(o[b][nt], a, pl[nt][0], pl[nt][1]);
                            }
                        }
                    }
                }
            }
        }

        // the lanes' row sums, and O in the units of V
        const float vs = Q8 ? v_ref * (1.0f / kWeightShift) : 1.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l[nt][x] += __shfl_xor_sync(FULL, l[nt][x], 4);
                l[nt][x] += __shfl_xor_sync(FULL, l[nt][x], 8);
                l[nt][x] += __shfl_xor_sync(FULL, l[nt][x], 16);
            }
        }
        const bool whole = last - first == n_tiles;
        if (active && whole) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = nt * 8 + 2 * tq + x;
                    if (r >= n_rows) continue;
                    const int i = r / p.gh;
                    const float f = vs / l[nt][x];
                    const size_t at = ((size_t)(q0 + i) * p.n_q_heads + (size_t)h * p.gh + r - i * p.gh) * D + gq * S::RL;
#pragma unroll
                    for (int run = 0; run < S::NRUN; ++run) {
#pragma unroll
                        for (int b = 0; b < S::RL / 2; ++b) {
                            const float a0 = o[run * (S::RL / 2) + b][nt][x] * f;
                            const float a1 = o[run * (S::RL / 2) + b][nt][2 + x] * f;
                            const size_t e = at + run * (D / S::NRUN) + 2 * b;
                            if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + e) = make_float2(a0, a1);
                            else *reinterpret_cast<uint32_t *>(static_cast<__half *>(p.out) + e) = pack2(a0, a1);
                        }
                    }
                }
            }
        } else if (active) {
            // A part: its record, then its arrival at the pair's counter.
            const long long i0 = sp.owner(ub), i1 = sp.owner(ub + n_tiles - 1);
            const size_t rec_row = (size_t)p.rows * REC;
            float *rec = p.recs + (((size_t)team * 2 + (first == 0 ? 1 : 0)) * p.hg + hl) * rec_row;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = nt * 8 + 2 * tq + x;
                    if (r >= n_rows) continue;
                    float *to = rec + (size_t)r * REC;
#pragma unroll
                    for (int run = 0; run < S::NRUN; ++run)
#pragma unroll
                        for (int b = 0; b < S::RL / 2; ++b)
                            *reinterpret_cast<float2 *>(to + gq * S::RL + run * (D / S::NRUN) + 2 * b) =
                                make_float2(o[run * (S::RL / 2) + b][nt][x] * vs, o[run * (S::RL / 2) + b][nt][2 + x] * vs);
                    if (gq == 0) *reinterpret_cast<float2 *>(to + D) = make_float2(m[nt][x], l[nt][x]);
                }
            }
            __syncwarp();
            int is_last = 0;
            if (lane == 0) {
                fence_acq_rel_gpu();
                // The counter holds (epoch, arrivals); any other epoch means none.
                unsigned long long *c = p.counters + (size_t)i0 * p.hg + hl;
                const unsigned long long stamp = (unsigned long long)p.epoch << 32;
                unsigned long long seen = 0, want;
                for (;;) {
                    want = (seen >> 32) == p.epoch ? seen + 1 : stamp + 1;
                    const unsigned long long old = atomicCAS(c, seen, want);
                    if (old == seen) break;
                    seen = old;
                }
                if ((long long)(want & 0xffffffffull) == i1 - i0 + 1) {
                    is_last = 1;
                    atomicExch(c, 0ull);
                }
                fence_acq_rel_gpu();
            }
            is_last = __shfl_sync(FULL, is_last, 0);
            if (is_last) {
                const int n_parts = (int)(i1 - i0) + 1;
                auto part = [&](int k) {   // the first part is the last pair of its team's span
                    return p.recs + (((size_t)(i0 + k) * 2 + (k == 0 ? 1 : 0)) * p.hg + hl) * rec_row;
                };
                constexpr int LPR = D / 4;         // lanes of a row, four dims each
                constexpr int WAYS = 32 / LPR;     // parts taken side by side
                const int way = lane / LPR, d4 = (lane % LPR) * 4;
                for (int r = 0; r < n_rows; ++r) {
                    float mm = kNoScore, ll = 0.0f;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int k0 = way; k0 < n_parts; k0 += 4 * WAYS) {
                        float4 a[4];
                        float2 ml[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            a[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            ml[k] = make_float2(kNoScore, 0.0f);
                            if (k0 + k * WAYS < n_parts) {
                                const float *from = part(k0 + k * WAYS) + (size_t)r * REC;
                                a[k] = __ldcg(reinterpret_cast<const float4 *>(from + d4));
                                ml[k] = __ldcg(reinterpret_cast<const float2 *>(from + D));
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float mn = fmaxf(mm, ml[k].x);
                            const float f0 = ex2(mm - mn), f1 = ex2(ml[k].x - mn);
                            acc.x = acc.x * f0 + a[k].x * f1;
                            acc.y = acc.y * f0 + a[k].y * f1;
                            acc.z = acc.z * f0 + a[k].z * f1;
                            acc.w = acc.w * f0 + a[k].w * f1;
                            ll = ll * f0 + ml[k].y * f1;
                            mm = mn;
                        }
                    }
                    if constexpr (WAYS == 2) {
                        const float mo = __shfl_xor_sync(FULL, mm, 16), lo = __shfl_xor_sync(FULL, ll, 16);
                        const float4 b = make_float4(__shfl_xor_sync(FULL, acc.x, 16), __shfl_xor_sync(FULL, acc.y, 16),
                                                     __shfl_xor_sync(FULL, acc.z, 16), __shfl_xor_sync(FULL, acc.w, 16));
                        const float mn = fmaxf(mm, mo);
                        const float f0 = ex2(mm - mn), f1 = ex2(mo - mn);
                        acc.x = acc.x * f0 + b.x * f1;
                        acc.y = acc.y * f0 + b.y * f1;
                        acc.z = acc.z * f0 + b.z * f1;
                        acc.w = acc.w * f0 + b.w * f1;
                        ll = ll * f0 + lo * f1;
                    }
                    if (way == 0) {
                        const int i = r / p.gh;
                        const float f = 1.0f / ll;
                        const size_t e = ((size_t)(q0 + i) * p.n_q_heads + (size_t)h * p.gh + r - i * p.gh) * D + d4;
                        if (p.out_f32)
                            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + e) =
                                make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
                        else
                            *reinterpret_cast<uint2 *>(static_cast<__half *>(p.out) + e) =
                                make_uint2(pack2(acc.x * f, acc.y * f), pack2(acc.z * f, acc.w * f));
                    }
                }
            }
        }
        // on to the next pair of the span
        cur.tile = cur.end - 1;
        advance(cur);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Kernel for this many rows per kv-head and output type.
using KernelFn = void (*)(Params);
struct Kernel {
    KernelFn fn;
    int smem;
};
template <typename T, int D>
Kernel pick(int n_rows, bool f32) {
    const int smem = Shape<T, D>::SMEM;
    if (n_rows <= 8)
        return {f32 ? rows_attention_kernel<T, D, 1, true> : rows_attention_kernel<T, D, 1, false>, smem};
    return {f32 ? rows_attention_kernel<T, D, 2, true> : rows_attention_kernel<T, D, 2, false>, smem};
}
Kernel kernel_e4m3(int head_dim, int n_rows, bool f32);   // rows_attention_e4m3.cu
Kernel kernel_f16(int head_dim, int n_rows, bool f32);    // rows_attention_f16.cu

}  // namespace rows
}  // namespace pkv
