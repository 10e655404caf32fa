// rows_attention.cuh -- attention of a few query rows per (sequence, kv-head)
// over the paged cache: decode and short appends over an e4m3 pool, short
// cross attention over either pool type.  (fp16 results of small batches with
// short tables, or with many rows, come from the prompt kernel.)
//
// For a (sequence s, kv-head h) with L tokens and at most 16 query rows (its
// query tokens x its gh q-heads, row r = i * gh + g of token i):
//   z_rt = scale * q_r . K_t,  out_r = sum_t softmax_t(z_r) V_t,
// t < L (cross, decode) or t <= L - n + i (causal), or what a window with sinks
// or a tree of drafts leaves (MASK; internal.h).  e4m3 pools: K_t = code *
// k_scale[page][h], V_t = code * v_scale[page][h].
//
// Floor: every K and V byte of the context is read once and used for at most 16
// rows, so it is HBM's.  Measured on GB300:
// 128 sequences of 16 to 2048 tokens, 12 heads x 64, e4m3 (93 MB) 24.0 us (26.6
// when the pool is not in L2), of which about 10 are the way to the first rows
// and the last merge; 256 sequences of 32 to 4096 tokens, 7 rows, 2 heads x 64
// (137 MB) 35.5 us; 16 x 2048 tokens, 40 heads x 128, fp32 results (336 MB) 63 us,
// 5.3 TB/s.  The first two are bound by latency and issue, not by HBM: 565 and
// 485 warp instructions per 4 KB stage, 45 % of the issue slots with four warps
// per scheduler.  Windows: 128 sequences of 32 to 16,384 tokens, window 1,024 and 4
// sinks, 7 rows, 2 heads x 64 18 us, 23.5 past L2 (67 MB); 16 of 4,096 to 8,192, 2,048 and 64, 40 heads x
// 128, e4m3, fp32 results 67 us, 5.2 TB/s.
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
// * Products on warp-level MMA m16n8k16 (fp16 in, fp32 sums) with the tokens
//   on the M side and the rows on the N side (8 columns): S^T = K Q^T and O^T =
//   V^T P^T, so up to 8 rows cost what one does.  The k order of the first is
//   free, so a lane reads 16-byte chunks of K rows as they lie; V is transposed
//   by ldmatrix.  e4m3 codes are widened to fp16 (exact) in between; V's
//   transpose is by bytes, and the token order of a tile is chosen so that a
//   lane's four tokens are two k pairs.  (Scores by mma.sync on e4m3 operands,
//   from three e4m3 terms of q, need no widening of K and were slower: 660
//   executed warp instructions per 4 KB stage by smsp__inst_executed, 574 with
//   the widening.)
// * Softmax in the log2 domain on the S^T fragments, fp32.  The running
//   maximum is raised only when a lane sees a score 2^8 above it, so its
//   reduction over the lanes is off the common path; the row sums stay per
//   lane until the end.
// * The K scale multiplies the score, the V scale the weight before it is
//   rounded to fp16 for the second product.  Weights are 2^7 times 2^(z - max)
//   (row sums too, so it cancels) and relative to the largest V scale met so
//   far: at most 2^15, and normal fp16 down to 2^-21 of the largest scale's.
//   The row sum is that of the fp32 weights.  fp32 output takes the product
//   twice, with the weight's fp16 part and with its rounding error, which is
//   normal fp16 down to 2^-10 of the largest scale's.  Below these a weight is
//   off by half of fp16's smallest, 2^-32 of the largest weight and scale.
// * A pair cut between spans leaves its parts (acc, m, l) in the workspace,
//   each with a flag that carries the launch's stamp, set behind one fence once
//   the warp's span is done; the warp of the pair's last part then waits for
//   the others' flags, merges the parts with the log-sum-exp rule and clears
//   the flags.  Every launch and replay has a stamp of its own, so a flag that
//   is set after a wait for it ran out counts for no later one.  The parts waited for belong to earlier spans, whose warps wait
//   for nothing but still earlier ones, and the wait is bounded (1 s).  Where
//   pairs are cut into many parts (few long contexts), the teams of a CTA merge
//   theirs first, behind a CTA barrier, and the CTAs' records are the parts.
#pragma once

#include <type_traits>

#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace rows {

constexpr int kMaxSeqs = 1024;       // sequences per launch
constexpr float kShiftLog2 = 7.0f;   // weights are 2^(z - m), m the maximum less this
constexpr float kRaiseLog2 = 15.0f;  // raise m when a weight would pass 2^15
constexpr float kNoScore = -1.0e30f; // m before any score
constexpr unsigned FULL = 0xffffffffu;

// Cost of a (sequence, group) pair in the partition, in stages: entering one
// costs a q load, a merge of lanes and a store.  (Measured with 1, 2, 4: the
// mixed batch of 128 sequences, 12 heads x 64, e4m3, 25.8, 24.1, 25.0 us.)
constexpr int kPairCost = 2;
// Least units per span: shorter ones cost more in merges than they bring.
// (Measured with 1, 2, 4, 8: 512 sequences of 32 tokens, 4 heads x 64, 7.6,
// 7.6, 9.9, 13.5 us; one of 2048 tokens, 40 heads x 128, 17.2, 17.1, 18.1,
// 21.4; 32 of up to 512 tokens, 4 rows, 13.6, 13.7, 13.4, 15.9.)
constexpr int kMinSpan = 2;
// With two levels.  (Measured with 2, 4, 6: 4 sequences of up to 4000 tokens, 8
// heads x 128, 20.0, 19.4, 20.3 us and, other lengths, 21.9, 18.4; 8 sequences,
// 4 rows x 64, 17.2, 18.3, 20.1.)
constexpr int kMinSpan2 = 4;
// A pair of n stages in spans of x takes x stages, then the merge of n / x
// parts, each kPartCost stages per 128 values of its rows: least at x =
// sqrt(kPartCost * values / 128 * n).
// (Measured with 0, 1/8, 1/4, 1/2: 6 sequences of 2,700 tokens, 4 rows, 128
// dims 28.6, 26.6, 29.8, 34.6 us; 14 of 1,600, 16 rows, 64 dims 24.6, 23.9,
// 25.5, 29.8.)
constexpr float kPartCost = 0.125f;
// More parts than this per longest pair: merged in two levels.  (Measured with
// 6, 12, 24 and one level only: 32 sequences of up to 512 tokens, 4 rows, 14.7,
// 13.4, 13.3, 13.4 us; 6 of 2,700 tokens, 4 rows x 128, 21.1, 21.0, 26.6, 26.6;
// one of 65,536 tokens, 4 rows x 128, 37.3, 37.4, 37.4, 88.6.)
constexpr float kMaxParts = 12.0f;
// A cut inside a pair of at most this many stages moves to the pair's nearer
// edge: such pairs stay whole and need no merge.  (Measured with 0, 4, 8 and
// spans of at least 4: 4 sequences of up to 100 tokens, 12 heads x 64, 11.7,
// 10.2, 10.3 us; larger batches the same within 1 %.)
constexpr int kWhole = 4;

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
    unsigned *flags;            // [team][2][head]: the stamp once that part's record is written
    float *recs;                // [team][2][head][rows][D + 4]: parts of cut pairs (acc, m, l)
    unsigned stamp;             // this launch's, 0 when it is captured (device_common.cuh)
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
    int after_append;       // the previous kernel wrote pages only: set out before it ends
    int out_f32;
    long long layer_row0;   // layer * n_blocks * block_size
    long long layer_page0;  // layer * n_blocks
    float scale_log2;
    AttnMask mask;
};

// PAGED: pages of 16 tokens and more, whose 16-token tiles lie in one page and
// have one scale; otherwise pages of one token.
template <typename T, int D, int NT, bool PAGED>
struct Shape {
    static constexpr bool Q8 = sizeof(T) == 1;
    static constexpr int RB = D * (int)sizeof(T);    // bytes of one head's row
    static constexpr int U = RB == 64 ? 2 : 1;       // 16-token tiles per stage
    static constexpr int ST = 16 * U;                // tokens per stage
    static constexpr int KV = ST * RB;               // K (or V) bytes of a stage
    static constexpr int SC = !Q8 ? 0 : (PAGED ? 16 : ST * 8);   // its scales: K, V per tile (K.., V.. per token)
    // warps per CTA (teams of 1, 2, 3 or 4): what registers and the ring allow
    static constexpr int NW = NT == 2 || RB == 256 ? 12 : 16;
    static constexpr int NST = RB == 256 ? 2 : 3;
    static constexpr int THREADS = 32 * NW;
    static constexpr int SMEM = NW * NST * (2 * KV + SC);
    static_assert(NW <= kFlagWarps, "the workspace's flags");
};

// Work units in order (sequence, group, stage): a pair has kPairCost units
// without work, then its stages.  W units are cut into n spans of q or (the
// first r) q + 1; team j takes [start(j), start(j + 1)), moved as kWhole says.
// W is below 2^31: the host bounds it by the tables.
struct Spans {
    unsigned n, q, r;
    unsigned T;   // teams that merge their parts of a pair before the others see them (1 or a CTA's)
    __device__ __forceinline__ unsigned start(unsigned j) const { return j * q + min(j, r); }
    // the span that holds unit x
    __device__ __forceinline__ unsigned owner(unsigned x) const {
        const unsigned big = r * (q + 1);
        return x < big ? x / (q + 1) : r + (x - big) / q;
    }
};

// Walks the stages of one team's span.
struct Cursor {
    int s;             // sequence; n_seqs: done
    int g;             // group
    int tile;          // next stage of the pair
    int end;           // one past the span's last stage of the pair
    int n_tiles;       // stages of the pair
};

// Two e4m3 codes (low or high half of w) to fp16, exact.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(w));
    return h;
}

// Two 16x16 byte matrices, transposed: lanes 16 i .. 16 i + 15 give the rows
// of matrix i; lane (g, t) receives column g of matrix i, rows 4t .. 4t + 3, in
// r[2 i], and column g + 8 in r[2 i + 1].
__device__ __forceinline__ void ldmatrix_b8_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
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
__device__ __forceinline__ float lds32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}

// Token p of a 16-token tile sits in row slot_of(p) of the MMA's M side.
// e4m3: lane t of a quad gets the transposed V of tokens 4t .. 4t + 3, of which
// the fp16 MMA takes 4t, 4t + 1 as k 2t, 2t + 1 and the others as k 2t + 8,
// 2t + 9, so these are the slots of the weights.  fp16: in order.
template <bool Q8>
__device__ __forceinline__ int slot_of(int p) {
    return Q8 ? ((p >> 1) & 1) * 8 + (p >> 2) * 2 + (p & 1) : p;
}
template <bool Q8>
__device__ __forceinline__ int token_of(int slot) {
    return Q8 ? ((slot >> 1) & 3) * 4 + (slot >> 3) * 2 + (slot & 1) : slot;
}

// Shared-memory offset of 16-byte chunk c of K slot r / V token r in a tile:
// chunks moved so that neither the 16-byte reads of K (eight lanes: two rows
// and four chunks) nor ldmatrix (eight rows, one chunk) meets a bank conflict.
template <int RB>
__device__ __forceinline__ uint32_t k_off(int r, int c) {
    return (uint32_t)(r * RB + ((RB == 64 ? c : c ^ ((r & 1) << 2)) << 4));
}
template <int RB>
__device__ __forceinline__ uint32_t v_off(int r, int c) {
    return (uint32_t)(r * RB + ((RB == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) << 4));
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

// MASK: a MaskKind.  A window's pair has the stages that hold a sink, then those
// from the first token of its first query's window on; stage i of the pair is
// stage i or i + skip of the context.  What no query of the pair sees is not
// read: rows are zero-filled, and blocks that hold only such tokens are not
// looked up.
template <typename T, int D, int NT, bool HILO, bool PAGED, int MASK>
__global__ void __launch_bounds__(Shape<T, D, NT, PAGED>::THREADS, 1) rows_attention_kernel(const Params p) {
    using S = Shape<T, D, NT, PAGED>;
    constexpr int NW = S::NW;
    constexpr int NTHREADS = S::THREADS;
    constexpr int RB = S::RB;
    constexpr int U = S::U;
    constexpr int ST = S::ST;
    constexpr int CPR = RB / 16;         // 16-byte chunks of a row
    constexpr int MT = D / 16;           // 16-dim tiles of O
    constexpr int REC = D + 4;           // floats of a row's record
    constexpr bool Q8 = S::Q8;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ unsigned pre[kMaxSeqs + 1];   // units before sequence s
    __shared__ int len_sh[kMaxSeqs];
    __shared__ int lo_sh[MASK == kMaskWindow ? kMaxSeqs : 1];   // first token that the first query sees by its window
    __shared__ unsigned warp_sum[32];
    __shared__ int warp_max[32];
    __shared__ Spans span_sh;
    __shared__ unsigned stamp_sh;

    const int warp = (int)threadIdx.x / 32;
    const int lane = (int)threadIdx.x % 32;

    // Launched as a programmatic dependent: everything below may read what the
    // stream's previous kernel wrote, or after a step's own append (which was
    // launched when everything before it had ended) the pages only.
    if (!p.after_append) griddep_wait();

    unsigned long long *count =          // of captured launches
        reinterpret_cast<unsigned long long *>(p.flags) - (kFlagOffset - kStateOffset) / sizeof(unsigned long long);
    if (warp == NW - 2 && lane == 0) stamp_sh = p.stamp ? p.stamp : count_stamp(ld_tagged(count) / kLaunchStep + 1);

    // The front of every table row into L2, shared out over the grid: the
    // lengths are not known yet.
    {
        const int lines = min((p.max_blocks * 4 + 127) / 128, 8);
        for (int e = (int)blockIdx.x * NTHREADS + (int)threadIdx.x; e < lines * p.n_seqs; e += (int)gridDim.x * NTHREADS)
            prefetch_l2(p.bt + (size_t)(e / lines) * p.max_blocks + e % lines * 32);
    }

    constexpr bool WINDOW = MASK == kMaskWindow, TREE = MASK == kMaskTree;
    // stages of a pair of sequence s (WINDOW: those with a sink of its L tokens, and the rest)
    auto sink_stages = [&](int L) { return (min(p.mask.sinks, L) + ST - 1) / ST; };
    auto n_stages = [&](int s) {
        const int L = len_sh[s], n = (L + ST - 1) / ST;
        if constexpr (WINDOW) return n - max(0, lo_sh[s] / ST - sink_stages(L));
        else return n;
    };

    // Prefix of the units over the sequences: each thread scans a run of
    // consecutive ones.
    {
        const int per = (p.n_seqs + NTHREADS - 1) / NTHREADS;
        const int s0 = min((int)threadIdx.x * per, p.n_seqs);
        const int s1 = min(s0 + per, p.n_seqs);
        unsigned mine = 0;
        int longest = 0;
        for (int s = s0; s < s1; ++s) {
            const int L = context_length(p, s, blockIdx.x == 0);
            len_sh[s] = L;
            if constexpr (WINDOW) {
                const int nq = p.cu_q ? min(p.cu_q[s + 1] - p.cu_q[s], p.rows / p.gh) : 1;
                lo_sh[s] = max(0, L - nq - p.mask.window + 1);
                longest = max(longest, n_stages(s) * ST);
            } else {
                longest = max(longest, L);
            }
            if (L > 0) mine += ((unsigned)n_stages(s) + kPairCost) * p.n_groups;
        }
        unsigned incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += x;
        }
        longest = __reduce_max_sync(FULL, longest);
        if (lane == 31) {
            warp_sum[warp] = incl;
            warp_max[warp] = longest;
        }
        __syncthreads();
        unsigned at = __reduce_add_sync(FULL, lane < warp ? warp_sum[lane] : 0u) + incl - mine;
        for (int s = s0; s < s1; ++s) {
            pre[s] = at;
            if (len_sh[s] > 0) at += ((unsigned)n_stages(s) + kPairCost) * p.n_groups;
        }
        if (warp == NW - 1) {
            longest = __reduce_max_sync(FULL, lane < NW ? warp_max[lane] : 0);
            if (lane == 31) {
                pre[p.n_seqs] = at;
                // few pairs: no more parts than pay (kPartCost)
                const float n_long = (float)((longest + ST - 1) / ST);
                const float cost = kPartCost * (float)((p.rows * D + 127) / 128) * n_long;
                const unsigned in_cta = NW / p.hg, teams = gridDim.x * in_cta;
                auto cut = [&](float c, int least_span) {
                    const unsigned least = max((unsigned)least_span, (unsigned)sqrtf(c));
                    return max(1u, min(teams, at / least));
                };
                unsigned n = cut(cost, kMinSpan), T = 1;
                if (in_cta > 1 && n_long * (float)n > kMaxParts * (float)at) {
                    T = in_cta;
                    n = cut(cost / (float)T, kMinSpan2);
                }
                span_sh = Spans{n, at / n, at % n, T};
            }
        }
        __syncthreads();
    }

    if (p.stamp == 0 && threadIdx.x == 0) add_launch(count);   // (stamp_sh has been read)

    // Rows of empty contexts: zeros.
    for (int s = (int)blockIdx.x * NW + warp; s < p.n_seqs; s += (int)gridDim.x * NW) {
        if (len_sh[s] > 0) continue;
        const int r0 = p.cu_q ? p.cu_q[s] : s;
        const int n = p.cu_q ? min(p.cu_q[s + 1] - r0, p.rows / p.gh) : 1;
        const size_t row = (size_t)p.n_q_heads * D;
        for (size_t e = lane; n > 0 && e < (size_t)n * row / 8; e += 32) {
            if (p.out_f32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + r0 * row) + 2 * e;
                o[0] = o[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            } else {
                reinterpret_cast<uint4 *>(static_cast<__half *>(p.out) + r0 * row)[e] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }

    const int hl = warp % p.hg;
    const unsigned team = blockIdx.x * (NW / p.hg) + warp / p.hg;
    const Spans sp = span_sh;
    if (warp / p.hg >= NW / p.hg || team >= sp.n || pre[p.n_seqs] == 0) {
        if (p.after_append) griddep_wait();   // this grid does not end before the append's
        return;
    }
    // The pair that holds unit x: its sequence and group, and x's distance from
    // the pair's first unit.
    auto pair_at = [&](unsigned x, int &s, int &g, unsigned &per) {
        // the last sequence with pre <= x: of 32 samples, then of 32 entries
        const int top = 32 * (__popc(__ballot_sync(FULL, lane * 32 < p.n_seqs && pre[lane * 32] <= x)) - 1);
        s = top + __popc(__ballot_sync(FULL, top + lane < p.n_seqs && pre[top + lane] <= x)) - 1;
        per = (unsigned)n_stages(s) + kPairCost;
        const unsigned d = x - pre[s];
        g = (int)(d / per);
        return d - (unsigned)g * per;
    };
    auto snapped = [&](unsigned x, int &s, int &g) {
        unsigned per;
        const unsigned d = pair_at(x, s, g, per);
        if (per > (unsigned)(kPairCost + kWhole)) return x;
        return 2 * d <= per ? x - d : x + per - d;
    };
    Cursor look;
    const unsigned u_lo = snapped(sp.start(team), look.s, look.g);
    unsigned u_hi = pre[p.n_seqs];
    if (team + 1 < sp.n) {
        int s, g;
        u_hi = snapped(sp.start(team + 1), s, g);
    }

    // Enter pair (c.s, c.g), or the next one of the span with a stage in it.
    auto settle = [&](Cursor &c) {
        for (;;) {
            while (c.s < p.n_seqs && len_sh[c.s] == 0) {
                ++c.s;
                c.g = 0;
            }
            if (c.s >= p.n_seqs) return;
            c.n_tiles = n_stages(c.s);
            const unsigned ub = pre[c.s] + (unsigned)c.g * (c.n_tiles + kPairCost) + kPairCost;   // its first stage
            if (ub >= u_hi) {
                c.s = p.n_seqs;
                return;
            }
            c.tile = u_lo > ub ? (int)(u_lo - ub) : 0;
            c.end = min(c.n_tiles, (int)(u_hi - ub));
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

    settle(look);
    Cursor cur = look;

    // --------------------------------------------------------------- copies
    const uint32_t ring = smem_addr(smem) + (uint32_t)warp * S::NST * 2 * S::KV;
    const uint32_t scales = smem_addr(smem) + (uint32_t)(NW * 2 * S::KV + warp * S::SC) * S::NST;
    const uint32_t tok_bytes = (uint32_t)p.n_kv_heads * RB;
    constexpr int PF = S::NST - 1;       // stages in flight, and stages looked up ahead
    constexpr int TI = 32 / CPR;         // tokens that the warp's lanes copy at once
    // this lane's chunk of the first TI tokens, and its place in a tile; the
    // next TI tokens are KSTEP slots and TI V rows further (v_off's swizzle
    // changes with them)
    const uint8_t *k_lane = p.k_pool + (size_t)(lane / CPR) * tok_bytes + (lane % CPR) * 16;
    const uint8_t *v_lane = p.v_pool + (size_t)(lane / CPR) * tok_bytes + (lane % CPR) * 16;
    const uint32_t k_at = ring + k_off<RB>(slot_of<Q8>(lane / CPR), lane % CPR);
    const uint32_t v_at = ring + S::KV + v_off<RB>(lane / CPR, lane % CPR);
    constexpr int KSTEP = Q8 ? TI / 2 : TI;
    auto v_xor = [](int i) { return RB == 64 ? 0u : (uint32_t)((i * TI) & 7) << 4; };
    // A stage to copy.  PAGED: lane l holds the block id of tile (l / 2) mod
    // U; otherwise that of token l mod ST.  What is not looked up has no id
    // (a table may hold any number): -2 there.
    struct Ahead {
        int id, tok0, h, n;              // first token, kv-head, tokens (0: nothing to copy)
        int lo, sinks;                   // WINDOW: of these the first, and those from lo on, are seen
    };
    Ahead ahead[PF];
    auto look_up = [&](Ahead &a) {
        a.n = 0;
        if (look.s >= p.n_seqs) return;
        a.tok0 = look.tile * ST;
        a.h = look.g * p.hg + hl;
        if (a.h < p.n_kv_heads) {        // the last group may have fewer heads
            const int L = len_sh[look.s];
            if constexpr (WINDOW) {
                if (look.tile >= sink_stages(L)) a.tok0 += ((L + ST - 1) / ST - look.n_tiles) * ST;
                a.lo = lo_sh[look.s] - a.tok0;
                a.sinks = p.mask.sinks - a.tok0;
            }
            a.n = min(ST, L - a.tok0);
            const int i = PAGED ? ((lane >> 1) & (U - 1)) * 16 : (lane & (ST - 1)), t = a.tok0 + i;
            bool seen = t < L;
            if constexpr (WINDOW) seen = seen && (i + (PAGED ? 15 : 0) >= a.lo || i < a.sinks);
            a.id = seen ? p.bt[(size_t)look.s * p.max_blocks + (PAGED ? t >> p.block_shift : t)] : -2;
        }
        advance(look);
    };
    auto copy = [&](int stage, const Ahead &a) {
        const uint32_t base = stage * 2 * S::KV;
        const uint32_t sc = scales + stage * S::SC;
        if (a.n > 0) {
            if constexpr (PAGED) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int id = __shfl_sync(FULL, a.id, 2 * u);
                    int left = a.n - 16 * u;
                    if ((unsigned)id >= (unsigned)p.n_blocks) {
                        const bool looked_up = left > 0 && (!WINDOW || 16 * u + 15 >= a.lo || 16 * u < a.sinks);
                        if (looked_up && lane == 0) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                        left = 0;
                    }
                    const bool whole = left >= 16 && (!WINDOW || 16 * u >= a.lo || 16 * u + 16 <= a.sinks);
                    const uint32_t kd = k_at + base + u * 16 * RB, vd = v_at + base + u * 16 * RB;
                    const unsigned row = (unsigned)p.layer_row0 + (unsigned)id * (unsigned)p.block_size +
                                         (unsigned)((a.tok0 + 16 * u) & (p.block_size - 1));   // below 2^31
                    const size_t at = (size_t)row * tok_bytes + (unsigned)(a.h * RB);
                    const uint8_t *ks = k_lane + at, *vs = v_lane + at;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 16 / TI; ++i) {
                            cp16(kd + i * KSTEP * RB, ks, 16u);
                            cp16((vd ^ v_xor(i)) + i * TI * RB, vs, 16u);
                            ks += TI * tok_bytes;
                            vs += TI * tok_bytes;
                        }
                    } else {   // rows past the context (that no query sees): zeros
#pragma unroll 1
                        for (int i = 0; i < 16 / TI; ++i) {
                            const int row_i = i * TI + lane / CPR;
                            const bool seen = !WINDOW || 16 * u + row_i >= a.lo || 16 * u + row_i < a.sinks;
                            const uint32_t n = row_i < left && seen ? 16u : 0u;
                            cp16(kd + i * KSTEP * RB, n ? ks : p.k_pool, n);
                            cp16((vd ^ v_xor(i)) + i * TI * RB, n ? vs : p.v_pool, n);
                            ks += TI * tok_bytes;
                            vs += TI * tok_bytes;
                        }
                    }
                }
                if constexpr (Q8) {
                    if (lane < 2 * U) {
                        const bool ok = (unsigned)a.id < (unsigned)p.n_blocks;
                        cp4(sc + lane * 4,
                            (lane & 1 ? p.v_scale : p.k_scale) + (ok ? (size_t)(p.layer_page0 + a.id) * p.n_kv_heads + a.h : 0),
                            ok ? 4u : 0u);
                    }
                }
            } else {
                const bool ok = (unsigned)a.id < (unsigned)p.n_blocks;
                const int i0 = lane & (ST - 1);
                if (!ok && i0 < a.n && (!WINDOW || i0 >= a.lo || i0 < a.sinks)) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                const int row = ok ? (int)(p.layer_row0 + a.id) : -1;
#pragma unroll
                for (int i = 0; i < ST / TI; ++i) {
                    const int r = __shfl_sync(FULL, row, i * TI + lane / CPR);
                    const uint32_t n = r < 0 ? 0u : 16u;
                    const size_t at = r < 0 ? 0 : (size_t)r * tok_bytes + a.h * RB + (lane % CPR) * 16;
                    const int u = i * TI / 16, iu = i % (16 / TI);
                    cp16(k_at + base + u * 16 * RB + iu * KSTEP * RB, p.k_pool + at, n);
                    cp16(((v_at + base) ^ v_xor(iu)) + u * 16 * RB + iu * TI * RB, p.v_pool + at, n);
                }
                if constexpr (Q8) {
                    const size_t at = ok ? (size_t)(p.layer_page0 + a.id) * p.n_kv_heads + a.h : 0;
                    if constexpr (ST == 32) {
                        cp4(sc + lane * 4, p.k_scale + at, ok ? 4u : 0u);
                        cp4(sc + ST * 4 + lane * 4, p.v_scale + at, ok ? 4u : 0u);
                    } else {
                        cp4(sc + lane * 4, (lane < ST ? p.k_scale : p.v_scale) + at, ok ? 4u : 0u);
                    }
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto look_further = [&]() {
#pragma unroll
        for (int k = 0; k + 1 < PF; ++k) ahead[k] = ahead[k + 1];
        look_up(ahead[PF - 1]);
    };
#pragma unroll
    for (int k = 0; k < PF; ++k) ahead[k].n = 0;
#pragma unroll 1
    for (int k = 0; k < PF; ++k) look_further();
    if (p.after_append) griddep_wait();
#pragma unroll 1
    for (int k = 0; k < PF; ++k) {
        copy(k, ahead[0]);
        look_further();
    }

    // ----------------------------------------------------------------- math
    const int gq = lane >> 2;            // N row of a B fragment, M row of an A fragment
    const int tq = lane & 3;
    const int tslot = token_of<Q8>(gq);  // token of slot gq; that of slot gq + 8:
    constexpr int SLOT8 = Q8 ? 2 : 8;    // SLOT8 further
    constexpr int KS = D / 16;           // k-steps of the scores
    const size_t rec_row = (size_t)p.rows * REC;
    int2 cut = make_int2(-1, 0);   // (sequence, group) of the pair that began in an earlier span
    bool goes_on = false;          // the last pair goes on in the next span
    int stage = 0;
    while (cur.s < p.n_seqs) {
        const int s = cur.s;
        const int h = cur.g * p.hg + hl;
        const bool active = h < p.n_kv_heads;
        const int L = len_sh[s];
        const int first = cur.tile, last = cur.end, n_tiles = cur.n_tiles;
        const unsigned ub = pre[s] + (unsigned)cur.g * (n_tiles + kPairCost) + kPairCost;
        const int q0 = p.cu_q ? p.cu_q[s] : s;
        const int nq = p.cu_q ? min(p.cu_q[s + 1] - q0, p.rows / p.gh) : 1;
        const int n_rows = nq * p.gh;

        // q as B fragments: lane (gq, tq) of a k-step holds dims of row gq in
        // the order in which it reads K: 16-byte chunks tq, tq + 4, ...
        uint32_t qb[KS][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + gq;
            const bool ok = active && r < n_rows;
            const int i = ok && nq > 1 ? r / p.gh : 0;
            const __half *src = p.q + ((size_t)(q0 + i) * p.n_q_heads + (size_t)(active ? h : 0) * p.gh +
                                       (ok ? r - i * p.gh : 0)) * D;
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
                vis[nt][e] = !TREE && p.causal && nq > 1 && r < n_rows ? max(0, L - nq + r / p.gh + 1) : L;
            }
        }
        if (p.causal) vis_min = max(0, L - nq + (TREE ? 0 : 1));
        int first_window = 0, skip = 0;  // WINDOW: the pair's first stage by the window, and how far it is moved
        int lo_max = 0;                  // the first token that the last query sees by its window
        if constexpr (WINDOW) {
            first_window = sink_stages(L);
            skip = (L + ST - 1) / ST - n_tiles;
            lo_max = L - p.mask.window;
        }
        uint32_t drafts[NT][2];          // TREE: those that rows 2 tq, 2 tq + 1 see
        if constexpr (TREE) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nt * 8 + 2 * tq + e;
                    drafts[nt][e] = r < n_rows ? (uint32_t)p.mask.tree[(size_t)(q0 + r / p.gh) * p.mask.tree_words] &
                                                     ((1u << nq) - 1u)
                                               : 0u;
                }
            }
        }

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
            copy(stage == 0 ? S::NST - 1 : stage - 1, ahead[0]);
            look_further();
            asm volatile("cp.async.wait_group %0;" ::"n"(PF) : "memory");
            __syncwarp();
            const uint32_t kb = ring + stage * 2 * S::KV;
            const uint32_t vb = kb + S::KV;
            const uint32_t scb = scales + stage * S::SC;
            stage = stage + 1 == S::NST ? 0 : stage + 1;
            if (!active) continue;

            // factors of the scores and of the weights, per slot gq, gq + 8
            // (PAGED: of the tile)
            constexpr int NSC = Q8 && !PAGED ? 2 : 1;
            float zf[U][NSC], vr[U][NSC];
            if constexpr (Q8) {
                float vm = 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int e = 0; e < NSC; ++e) {
                        // (above 0, so that a masked -inf stays one)
                        zf[u][e] = fmaxf(lds32(scb + (PAGED ? 2 * u : u * 16 + e * SLOT8 + tslot) * 4) * p.scale_log2, 1e-37f);
                        vr[u][e] = lds32(scb + (PAGED ? 2 * u + 1 : ST + u * 16 + e * SLOT8 + tslot) * 4);
                        vm = fmaxf(vm, vr[u][e]);
                    }
                }
                if constexpr (!PAGED) vm = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(vm)));   // (not negative)
                if (vm > v_ref) {
                    const float f = v_ref / vm;
                    v_ref = vm;
                    v_inv = 1.0f / vm;
#pragma unroll
                    for (int b = 0; b < MT; ++b)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[b][nt][e] *= f;
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < NSC; ++e) vr[u][e] *= v_inv;
            } else {
                zf[0][0] = p.scale_log2;
            }

            // products of slots gq and gq + 8 with rows 2 tq, 2 tq + 1
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
                    constexpr int STEPS = Q8 ? 4 : 2;   // k-steps of a chunk
#pragma unroll
                    for (int w = 0; w < STEPS; ++w) {
                        uint32_t a[4];
                        if constexpr (Q8) {
                            a[0] = widen_lo(wa[w]);
                            a[1] = widen_lo(wc[w]);
                            a[2] = widen_hi(wa[w]);
                            a[3] = widen_hi(wc[w]);
                        } else {
                            a[0] = wa[2 * w];
                            a[1] = wc[2 * w];
                            a[2] = wa[2 * w + 1];
                            a[3] = wc[2 * w + 1];
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(z[u][nt], a, qb[i * STEPS + w][nt][0], qb[i * STEPS + w][nt][1]);
                    }
                }
            }
            const int tok0 = (tile + (WINDOW && tile >= first_window ? skip : 0)) * ST;
            if constexpr (WINDOW) {      // before the window of some row, and no sink
                if (tok0 < lo_max && tok0 + ST > p.mask.sinks) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int t = tok0 + u * 16 + (e >> 1) * SLOT8 + tslot;
                                if (t < vis[nt][e & 1] - p.mask.window && t >= p.mask.sinks) z[u][nt][e] = -INFINITY;
                            }
                }
            }
            if constexpr (TREE) {
                if (tok0 + ST > vis_min) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int d = tok0 + u * 16 + (e >> 1) * SLOT8 + tslot - (L - nq);   // draft
                                if (d >= 0 && (d >= 32 || !(drafts[nt][e & 1] >> (d & 31) & 1u))) z[u][nt][e] = -INFINITY;
                            }
                }
            }
            if (!TREE && tok0 + ST > vis_min) {   // the context's end, or a causal limit
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (tok0 + u * 16 + (e >> 1) * SLOT8 + tslot >= vis[nt][e & 1]) z[u][nt][e] = -INFINITY;
            }
            float mx[NT][2];             // log2 scores' maxima (the factors are positive)
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float v = NSC == 2 ? fmaxf(z[u][nt][x] * zf[u][0], z[u][nt][2 + x] * zf[u][NSC - 1])
                                                 : fmaxf(z[u][nt][x], z[u][nt][2 + x]) * zf[u][0];
                        mx[nt][x] = u == 0 ? v : fmaxf(mx[nt][x], v);
                    }
                    raise |= mx[nt][x] > m[nt][x] + kRaiseLog2;
                }
            }
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
                            const float f = ex2(m[nt][x] - (v - kShiftLog2));
                            m[nt][x] = v - kShiftLog2;
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
                        const float f = zf[u][NSC == 2 ? e : 0];
                        float w0 = ex2(fmaf(z[u][nt][2 * e], f, -m[nt][0]));
                        float w1 = ex2(fmaf(z[u][nt][2 * e + 1], f, -m[nt][1]));
                        l[nt][0] += w0;
                        l[nt][1] += w1;
                        if constexpr (Q8) {
                            w0 *= vr[u][NSC == 2 ? e : 0];
                            w1 *= vr[u][NSC == 2 ? e : 0];
                        }
                        const uint32_t hi = pack2(w0, w1);
                        pb[nt][e] = transpose8x8(hi);
                        if constexpr (HILO) {
                            const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                            pl[nt][e] = transpose8x8(pack2(w0 - hf.x, w1 - hf.y));
                        }
                    }
                }
                // O^T += V^T P^T, 16 dims at a time (e4m3: 32 per load).  fp32
                // output sums each tile apart and adds it rounded: the MMA's
                // own accumulation drops what lies below its largest term.
                auto product = [&](int b, const uint32_t (&a)[4]) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (HILO) {
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16_16816(d, a, pl[nt][0], pl[nt][1]);
                            mma_f16_16816(d, a, pb[nt][0], pb[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[b][nt][e] += d[e];
                        } else {
                            mma_f16_16816(o[b][nt], a, pb[nt][0], pb[nt][1]);
                        }
                    }
                };
                if constexpr (Q8) {
#pragma unroll
                    for (int c = 0; c < CPR; c += 2) {
                        uint32_t r[4];
                        ldmatrix_b8_trans(r, vb + u * 16 * RB + v_off<RB>(lane & 15, c + (lane >> 4)));
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t a[4] = {widen_lo(r[2 * k]), widen_lo(r[2 * k + 1]), widen_hi(r[2 * k]),
                                                   widen_hi(r[2 * k + 1])};
                            product(c + k, a);
                        }
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < MT; ++b) {
                        uint32_t a[4];
                        ldmatrix_x4_trans(a, vb + u * 16 * RB + v_off<RB>((lane & 7) + (lane >> 4) * 8, 2 * b + ((lane >> 3) & 1)));
                        product(b, a);
                    }
                }
            }
        }

        // the lanes' row sums, and O in the units of V
        const float vs = Q8 ? v_ref : 1.0f;
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
        // Lanes of neighbouring gq swap halves, so that each stores two
        // neighbouring dims of one row: row nt * 8 + 2 tq + (gq & 1).
        auto each_pair = [&](const float (&f)[NT][2], auto store) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int b = 0; b < 2 * MT; ++b) {
                    const float v0 = o[b / 2][nt][2 * (b & 1)] * f[nt][0], v1 = o[b / 2][nt][2 * (b & 1) + 1] * f[nt][1];
                    const float got = __shfl_xor_sync(FULL, gq & 1 ? v0 : v1, 4);
                    store(nt, b * 8 + (gq & 6), gq & 1 ? make_float2(got, v1) : make_float2(v0, got));
                }
            }
        };
        if (active && whole) {
            float f[NT][2];
            size_t at[NT];
            bool ok[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // (a draft may see nothing at all: zeros)
                f[nt][0] = TREE && l[nt][0] == 0.0f ? 0.0f : vs / l[nt][0];
                f[nt][1] = TREE && l[nt][1] == 0.0f ? 0.0f : vs / l[nt][1];
                const int r = nt * 8 + 2 * tq + (gq & 1);
                const int i = nq > 1 ? r / p.gh : 0;
                ok[nt] = r < n_rows;
                at[nt] = ((size_t)(q0 + i) * p.n_q_heads + (size_t)h * p.gh + r - i * p.gh) * D;
            }
            each_pair(f, [&](int nt, int d, float2 v) {
                if (!ok[nt]) return;
                if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at[nt] + d) = v;
                else *reinterpret_cast<uint32_t *>(static_cast<__half *>(p.out) + at[nt] + d) = pack2(v.x, v.y);
            });
        } else if (active) {
            // A part: its record (slot 1 of the team for the pair's first part).
            const int slot = first == 0 ? 1 : 0;
            float *rec = p.recs + (((size_t)team * 2 + slot) * p.hg + hl) * rec_row;
            if (slot == 0) cut = make_int2(s, cur.g);
            else goes_on = true;
            float f[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) f[nt][0] = f[nt][1] = vs;
            each_pair(f, [&](int nt, int d, float2 v) {
                const int r = nt * 8 + 2 * tq + (gq & 1);
                if (r < n_rows) *reinterpret_cast<float2 *>(rec + (size_t)r * REC + d) = v;
            });
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = nt * 8 + 2 * tq + gq;
                if (gq < 2 && r < n_rows)
                    *reinterpret_cast<float2 *>(rec + (size_t)r * REC + D) =
                        gq ? make_float2(m[nt][1], l[nt][1]) : make_float2(m[nt][0], l[nt][0]);
            }
        }
        // on to the next pair of the span
        cur.tile = cur.end - 1;
        advance(cur);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    const bool group_end = team % sp.T == sp.T - 1;
    unsigned ub = 0, team0 = 0;          // the pair that began earlier: first stage's unit, first team
    bool ends = false;                   // its last part is here
    if (cut.x >= 0) {
        const unsigned n_tiles = (unsigned)n_stages(cut.x);
        ub = pre[cut.x] + (unsigned)cut.y * (n_tiles + kPairCost) + kPairCost;
        ends = ub + n_tiles <= u_hi;
    }
    auto flag_parts = [&](bool slot0, bool slot1) {   // these records are for others to read
        if (!slot0 && !slot1) return;
        __syncwarp();
        if (lane == 0) {
            fence_acq_rel_gpu();
            if (slot0) st_relaxed(p.flags + team * 2 * p.hg + hl, stamp_sh);
            if (slot1) st_relaxed(p.flags + (team * 2 + 1) * p.hg + hl, stamp_sh);
        }
    };
    flag_parts(sp.T == 1 && cut.x >= 0 && !ends, goes_on && group_end);
    if (sp.T > 1) __syncthreads();       // the CTA's records are written
    if (cut.x < 0 || (!ends && (sp.T == 1 || !group_end))) return;   // (!ends: the CTA's last team merges it)

    // The pair that began in an earlier span: merge its parts, first the
    // CTA's, when this is the last of them, then, when this is the pair's last
    // part, the CTAs' (T = 1: there is no first step).  What another SM wrote
    // takes about 1.2 us to arrive and a lone warp issues an instruction every
    // few cycles, so the loads of a step go out together and few instructions
    // lie between: a lane takes ITEMS (row, four dims) items of AHEAD parts, 16
    // loads in all.
    __syncwarp();
    team0 = sp.owner(ub);
    const unsigned from0 = sp.T == 1 ? team : max(team0, team - team % sp.T);
    const unsigned group0 = sp.T == 1 ? team0 : team0 / sp.T, group = sp.T == 1 ? team : team / sp.T;
    const int h = cut.y * p.hg + hl;
    const int q0 = p.cu_q ? p.cu_q[cut.x] : cut.x;
    const int nq = p.cu_q ? min(p.cu_q[cut.x + 1] - q0, p.rows / p.gh) : 1;
    const int n_rows = nq * p.gh;
#pragma unroll 1
    for (int level = from0 == team ? 1 : 0; level < 2; ++level) {   // (one part of the CTA: as it is)
    // Part k of this level lies with this team (teams from0 .. this one, or the
    // last team of each CTA that has a part): in slot 1 of the pair's first.
    const int n_parts = (int)(level == 0 ? team - from0 : group - group0) + 1;
    const unsigned u0 = level == 0 ? from0 : group0 * sp.T + sp.T - 1, step = level == 0 ? 1 : sp.T;
    auto place = [&](int k) {
        const unsigned u = min(team, u0 + k * step);
        return (u * 2 + (u == team0 ? 1 : 0)) * p.hg + hl;
    };
    const bool last_level = level == 1 || (ends && from0 == team0);
    if (level == 1) {
        unsigned long long since = 0;
        for (int k0 = 0; k0 < n_parts - 1; k0 += 32) {
            unsigned *flag = p.flags + place(min(k0 + lane, n_parts - 2));
            while (!__all_sync(FULL, ld_acquire(flag) == stamp_sh)) {
                const unsigned long long now = global_timer_ns();
                if (since == 0) since = now;
                if (__any_sync(FULL, now - since > kWaitLimitNs)) {
                    if (lane == 0) atomicOr(p.status, PF_DEV_WAIT_TIMEOUT);
                    return;
                }
            }
            __syncwarp();
            if (k0 + lane < n_parts - 1) st_relaxed(flag, 0u);
        }
    }
    // the warp's ring now holds (m, l), then (factor, l), of a chunk of parts
    constexpr int CHUNK = 480;
    float2 *ml = reinterpret_cast<float2 *>(smem + (size_t)warp * S::NST * 2 * S::KV);   // [part][row]
    float *sum_l = reinterpret_cast<float *>(ml + CHUNK);   // [16], then [16] maxima
    static_assert(CHUNK * 8 + 128 + NT * 8 * D * 4 <= S::NST * 2 * S::KV, "the ring holds the merge's tables");
    float *sum = sum_l + 32;                 // [rows][D], when there are several chunks
    const int per = min(n_parts, CHUNK / n_rows);
    if (lane < 16) {
        sum_l[lane] = 0.0f;
        sum_l[16 + lane] = kNoScore;
    }
    __syncwarp();
    constexpr int LPR = D / 4;
    const int items = n_rows * LPR;
    for (int p0 = 0; p0 < n_parts; p0 += per) {
        const int np = min(per, n_parts - p0);
        const bool only = per == n_parts, final_chunk = p0 + np == n_parts;
        // each row's maximum and sum: groups of LW lanes share a row's parts
        const int LW = n_rows <= 2 ? 16 : (n_rows <= 4 ? 8 : (n_rows <= 8 ? 4 : 2));
        {
            const int r = min(lane / LW, n_rows - 1), k1 = lane % LW;
            const float old = sum_l[16 + r];
            float mn = old;
            for (int k = k1; k < np; k += 4 * LW) {
                float2 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = __ldcg(reinterpret_cast<const float2 *>(p.recs + place(p0 + min(k + i * LW, np - 1)) * rec_row + r * REC + D));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mn = fmaxf(mn, v[i].x);
                    if (k + i * LW < np && lane / LW < n_rows) ml[(k + i * LW) * n_rows + r] = v[i];
                }
            }
            for (int o = LW / 2; o; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(FULL, mn, o));
            float ls = 0.0f;
            for (int k = k1; k < np && lane / LW < n_rows; k += LW) {
                float2 &v = ml[k * n_rows + r];
                v.x = ex2(v.x - mn);
                ls = fmaf(v.y, v.x, ls);
            }
            for (int o = LW / 2; o; o >>= 1) ls += __shfl_xor_sync(FULL, ls, o);
            __syncwarp();
            if (k1 == 0 && lane / LW < n_rows) {
                sum_l[r] = fmaf(sum_l[r], ex2(old - mn), ls);
                sum_l[16 + r] = mn;
            }
            if (p0 > 0) {                    // earlier chunks' sums to the new maximum
                const float g = ex2(old - mn);
                for (int q = 0; q < n_rows; ++q) {
                    const float f = __shfl_sync(FULL, g, q * LW);
                    for (int d = lane; d < D; d += 32) sum[q * D + d] *= f;
                }
            }
            __syncwarp();
        }
        auto combine = [&](auto items_c, auto ahead_c) {
        constexpr int ITEMS = decltype(items_c)::value, AHEAD = decltype(ahead_c)::value;
        for (int e0 = 0; e0 < items; e0 += 32 * ITEMS) {
            float4 acc[ITEMS];
            const float *at[ITEMS];
            int row[ITEMS];
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int e = min(e0 + i * 32 + lane, items - 1);
                row[i] = e / LPR;
                at[i] = p.recs + row[i] * REC + (e % LPR) * 4;
                acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            for (int k0 = 0; k0 < np; k0 += AHEAD) {
                float4 a[ITEMS][AHEAD];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const size_t off = place(p0 + min(k0 + k, np - 1)) * rec_row;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) a[i][k] = __ldcg(reinterpret_cast<const float4 *>(at[i] + off));
                }
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    if (k0 + k >= np) break;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) {
                        const float f = ml[(k0 + k) * n_rows + row[i]].x;
                        acc[i].x = fmaf(a[i][k].x, f, acc[i].x);
                        acc[i].y = fmaf(a[i][k].y, f, acc[i].y);
                        acc[i].z = fmaf(a[i][k].z, f, acc[i].z);
                        acc[i].w = fmaf(a[i][k].w, f, acc[i].w);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int e = e0 + i * 32 + lane;
                if (e >= items) break;
                const int d4 = (e % LPR) * 4;
                float4 &s4 = *reinterpret_cast<float4 *>(sum + row[i] * D + d4);
                if (p0 > 0) acc[i] = make_float4(acc[i].x + s4.x, acc[i].y + s4.y, acc[i].z + s4.z, acc[i].w + s4.w);
                if (!only && !final_chunk) {
                    s4 = acc[i];
                    continue;
                }
                if (!last_level) {       // in place of the last part's (whose items no other lane reads)
                    *reinterpret_cast<float4 *>(p.recs + place(n_parts - 1) * rec_row + row[i] * REC + d4) = acc[i];
                    continue;
                }
                const int j = nq > 1 ? row[i] / p.gh : 0;
                const float f = TREE && sum_l[row[i]] == 0.0f ? 0.0f : 1.0f / sum_l[row[i]];
                const size_t o = ((size_t)(q0 + j) * p.n_q_heads + (size_t)h * p.gh + row[i] - j * p.gh) * D + d4;
                if (p.out_f32)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + o) =
                        make_float4(acc[i].x * f, acc[i].y * f, acc[i].z * f, acc[i].w * f);
                else
                    *reinterpret_cast<uint2 *>(static_cast<__half *>(p.out) + o) =
                        make_uint2(pack2(acc[i].x * f, acc[i].y * f), pack2(acc[i].z * f, acc[i].w * f));
            }
        }
        };
        if (items <= 32) combine(std::integral_constant<int, 1>(), std::integral_constant<int, 16>());
        else combine(std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
        __syncwarp();
    }
    if (last_level) return;
    if (lane < n_rows)
        *reinterpret_cast<float2 *>(p.recs + place(n_parts - 1) * rec_row + lane * REC + D) =
            make_float2(sum_l[16 + lane], sum_l[lane]);
    __syncwarp();
    if (!ends) {
        flag_parts(true, false);
        return;
    }
    }
}

// Kernel for this many rows per kv-head, output type and page size.
using KernelFn = void (*)(Params);
struct Kernel {
    KernelFn fn;
    int smem;
    int warps;
};
template <typename T, int D, int MASK, int NT, bool PAGED>
Kernel instance(bool f32) {
    return {f32 ? rows_attention_kernel<T, D, NT, true, PAGED, MASK> : rows_attention_kernel<T, D, NT, false, PAGED, MASK>,
            Shape<T, D, NT, PAGED>::SMEM, Shape<T, D, NT, PAGED>::NW};
}
template <typename T, int D, int MASK = kMaskNone>
Kernel pick(int n_rows, bool f32, bool paged) {
    if (n_rows <= 8) return paged ? instance<T, D, MASK, 1, true>(f32) : instance<T, D, MASK, 1, false>(f32);
    return paged ? instance<T, D, MASK, 2, true>(f32) : instance<T, D, MASK, 2, false>(f32);
}
// one file each: rows_attention_<type>_d<head_dim>.cu, and with a mask
// rows_attention_<type>_d<head_dim>_<mask>.cu
Kernel kernel_e4m3_d64(int n_rows, bool f32, bool paged);
Kernel kernel_e4m3_d128(int n_rows, bool f32, bool paged);
Kernel kernel_f16_d64(int n_rows, bool f32, bool paged);
Kernel kernel_f16_d128(int n_rows, bool f32, bool paged);
Kernel kernel_e4m3_d64_window(int n_rows, bool f32, bool paged);
Kernel kernel_e4m3_d128_window(int n_rows, bool f32, bool paged);
Kernel kernel_f16_d64_window(int n_rows, bool f32, bool paged);
Kernel kernel_f16_d128_window(int n_rows, bool f32, bool paged);
Kernel kernel_e4m3_d64_tree(int n_rows, bool f32, bool paged);
Kernel kernel_e4m3_d128_tree(int n_rows, bool f32, bool paged);
Kernel kernel_f16_d64_tree(int n_rows, bool f32, bool paged);
Kernel kernel_f16_d128_tree(int n_rows, bool f32, bool paged);

}  // namespace rows
}  // namespace pkv
