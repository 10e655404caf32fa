// prompt_masked.cuh -- attention of many query rows under a mask over the paged
// cache, on the fifth-generation tensor cores: pf_paged_window_attention and
// pf_paged_tree_attention (more than 16 rows per kv-head, and small batches of
// fewer).
//
// A kv-head's query rows are its sequence's n new tokens x its gh q-heads, row
// r = i * gh + g.  A block is 256 consecutive rows of one (sequence, kv-head),
// two query tiles of 128 (the MMA's M); with long contexts of few blocks
// (SPLIT) also one part of the context, whose parts merge_masked_kernel joins.
//
// What a block walks is counted in virtual tokens.  Tree: the context.  Window:
// the boxes (units that are looked up and copied together: what a page holds of
// a tile) with a sink, then, moved down to them, those from the first token that
// the block's first row sees by its window on:
//   context token of virtual token x = x + (x < sink_end ? 0 : skip),
// so that sinks and window share tiles, every box holds a token that the block
// sees, and blocks that no query sees are not looked up.  A row at virtual position
// lim sees x <= lim with x > lim - window or x < sinks.
//
// The CTAs stay: one per SM, which takes every grid-th block (to and fro, the
// longest first), and its sixteen warps run through the blocks on their own,
// held together by mbarriers:
//   warps 0-3 and 4-7  the softmax of query tile 0 and 1 (thread t: row t, lane t
//                      of tensor memory), its output, and the next block's query
//                      rows, once the last scores of this one are done;
//   warps 8-11         the loaders, two for K and two for V, into a ring of NS
//                      stages that goes on from block to block;
//   warps 12, 13       one elected thread each issues the scores S_g = Q_g K_j^T
//                      and the products O_g += P_g V_j;
//   warp 14            what the next blocks are, up to kInfos ahead (15 idles).
// So a block's first tiles, its query rows and its first scores are there when
// the block before is written.
//
// Calls of at most 128 rows per (sequence, kv-head) (DUAL) have one query tile a
// block: the two groups of softmax warps take its even and its odd tiles, each
// with a maximum, a sum and an O of its own, and join them at the block's end, half
// of the dims each.  64 tokens (a tile at head_dim 128, half of one at 64), 16 blocks
// that stay in L2: fp16 x 128 0.56 us, 0.76 with both query tiles; fp16 x 64 0.33 and
// 0.62; e4m3 x 128 0.73 and 0.99.
//
// Per tile (see prefill_tc.cu): scores in tensor memory, a running maximum per row
// in the log2 domain that is raised only past 2^8, weights rounded to fp16 into
// tensor memory, row sums of the fp32 weights.  A row may see nothing of a tile, of
// a part or (tree) at all: its maximum stays -inf, its sum 0, its output zeros.
//
// Measured (GB300; 4 prompts of 4,096 tokens, 32 q-heads over 8 kv-heads x 128,
// window 512, 4 sinks): 142 us in a CUDA graph, 902 TFLOP/s (146 on another board), tensor
// pipe busy 47 % of the cycles; over an 8-bit pool 184, over fp16 pages of one token 209
// (a tile's copies are waited for before the next tile's).  A CTA per block took 205, of
// which 6.4 us a block beside 0.76 us a tile (blocks of 4, 10 and 18 tiles): the chain lengths, block
// ids, rows, scores, weights, product, output, of which nothing overlapped.  Two
// CTAs of 128 rows per SM instead took 198 (each is such a chain).  Here the query
// rows fetched by warps of their own took 203, by the softmax warps 168; with the
// blocks' lengths and divisions left to warp 14, and query tile 0 read from tensor
// memory, 140.  The latter fits a bound by shared memory at head_dim 128: with
// 64 tokens on the N side an MMA of the scores reads 6 KB for 32 cycles of products,
// and a tile moved 160 KB, 1,280 cycles at 128 bytes; it took 1,300.  Two softmax
// warps per 32 rows were slower (188).  Trees of 100 to 200 drafts (8 sequences of
// 1,024 to 2,048 tokens, 40 heads x 128): 60 us, 4.6 TB/s, 69.9 before CTAs
// that take a block more took the short ones.
#pragma once

#include <type_traits>

#include "internal.h"
#include "tcgen05.cuh"

namespace pkv {
namespace prompt_masked {

using namespace prefill_tc;   // tcgen05.cuh

constexpr int QT = 128;            // rows per query tile (the MMA's M)
constexpr int ROWS = 2 * QT;       // of a block
constexpr int NTHREADS = 512;
constexpr int SOFTMAX_WARPS = 8;
constexpr int LOAD_WARP0 = 8;      // K loaders (warps 8, 9), V loaders (10, 11)
constexpr int MMA_S_WARP = 12;     // owns the tensor memory
constexpr int MMA_PV_WARP = 13;
constexpr int INFO_WARP = 14;      // (15 idles)
constexpr int kMinTiles = 4;       // of a part
constexpr int kMaxParts = 32;      // a lane each in the merge
constexpr int kOrderSeqs = 256;    // sequences that a CTA puts in order (a byte each)
constexpr int kOrderContext = 1024;
constexpr int kInfos = 4;
constexpr int TMEM_COLS = 512;
constexpr float kRescaleLog2 = 8.0f;

// Registers: as many softmax threads as others, launched with 128 each.
template <int D>
struct Regs {
    static constexpr int SOFTMAX = D == 64 ? 200 : 152;
    static constexpr int OTHER = 256 - SOFTMAX;
    static_assert(SOFTMAX % 8 == 0 && 2 * 128 * (SOFTMAX + OTHER) == NTHREADS * 128, "the split is the launch's registers");
};

template <int D, bool Q8, bool DUAL>
struct Cfg {
    static constexpr int NS = Q8 ? 3 : 4;               // K/V stages
    static constexpr int RAW = 2;                       // e4m3: stages of codes (more, up to 5, changed nothing)
    static constexpr int BN = D == 64 ? 128 : 64;       // tokens per K/V tile (the scores' N)
    static constexpr int HALVES = D / 64;               // 64-element halves of a row
    static constexpr int Q_BYTES = QT * D * 2;          // one query tile
    static constexpr int KV_BYTES = BN * D * 2;         // one K or V tile
    static constexpr int OUT_BYTES = 32 * 128;          // a softmax warp's rows on their way out
    static constexpr int OFF_K = (DUAL ? 1 : 2) * Q_BYTES;
    static constexpr int OFF_V = OFF_K + NS * KV_BYTES;
    static constexpr int OFF_OUT = OFF_V + NS * KV_BYTES;
    static constexpr int OFF_RAW = OFF_OUT + SOFTMAX_WARPS * OUT_BYTES;
    static constexpr int RAW_BYTES = Q8 ? BN * D + BN * 4 : 0;   // codes of a K or V tile, then the scales of its tokens
    static constexpr int OFF_ML = OFF_RAW + 2 * RAW * RAW_BYTES;   // DUAL: maxima and sums of both groups
    static constexpr int DATA = OFF_ML + (DUAL ? 2 * QT * 8 : 0);
    static constexpr int SMEM = DATA + 1024;            // slack to align the base to 1024 bytes
    // tensor memory (fp32 columns): S, O, and P (two weights per column) of both tiles
    static constexpr int COL_O = 2 * BN;
    static constexpr int COL_P = COL_O + 2 * D;
    // head_dim 128: the query rows of tile 0 (two values per column), which its
    // scores take from there
    static constexpr bool Q0_TMEM = D == 128;
    static constexpr int COL_Q = COL_P + BN;
    static_assert(COL_Q + (Q0_TMEM ? D / 2 : 0) <= TMEM_COLS, "tensor memory columns");
};

struct Params {
    const __half *q;
    const void *k_pool;
    const void *v_pool;
    const float *k_scale;   // e4m3 pools
    const float *v_scale;
    void *out;
    const int32_t *bt;
    const int32_t *lens;
    const int32_t *cu_q;    // null (window): one query per sequence, row s
    int *status;
    int n_q_heads;
    int n_kv_heads;
    int gh;
    int gh_magic;     // 65536 / gh, rounded up
    int max_blocks;
    int max_new;
    int n_blocks;
    int block_size;
    int block_shift;  // log2 of block_size
    int unit_shift;   // log2 of the rows copied together
    int n_seqs;
    int n_items;      // sequences x kv-heads
    int n_qp;         // blocks of rows of the longest (sequence, kv-head)
    int n_work;       // blocks x parts
    long long layer_row0;
    long long layer_page0;   // layer * n_blocks
    int out_f32;
    float scale_log2;
    AttnMask mask;
    unsigned long long wait_ns;   // of any wait on chip
    int splits;       // parts at most
    float2 *part_ml;  // [block][part][ROWS]: a row's reference maximum (log2) and sum of weights
    float *part_o;    // [block][part][ROWS][D]: its sum of weighted values
};

// Tiles of a part when a block's n tiles are cut into at most `splits`.
__device__ __forceinline__ int part_tiles(int n, int splits) { return max(kMinTiles, (n + splits - 1) / splits); }

// What the call says of a sequence: its length, first and one past the last query row.
struct Seq {
    int L, q0, q1;
};

// A block: rows r0 .. r_end - 1 of a (sequence, kv-head), and what they see.
template <int BN, int MASK>
struct Block {
    int L, q0, n;             // clamped
    int r0, r_end;
    int base;                 // position of new token 0
    int lim[2];               // per query tile: its last virtual position (-1: no row)
    int last;                 // the block's
    int sinks, sink_end, skip;
    int lo;                   // virtual tokens sinks .. lo - 1 are seen by no row
    int tiles;

    // bad: the call does not allow these lengths
    __device__ __forceinline__ void make(const Params &p, const Seq &seq, int qp, bool &bad) {
        constexpr bool WINDOW = MASK == kMaskWindow;
        const int most = p.max_blocks << p.block_shift;
        bad = false;
        L = seq.L;
        if (L < 0 || L > most) {
            bad = true;
            L = L < 0 ? 0 : most;
        }
        q0 = seq.q0;
        n = seq.q1 - seq.q0;
        const bool step = WINDOW && !p.cu_q;
        if (!step && (n < 0 || n > L || n > p.max_new)) {
            bad = true;
            n = n < 0 ? 0 : min(min(n, L), p.max_new);
        }
        const int rows = n * p.gh;
        r0 = qp * ROWS;
        r_end = min(r0 + ROWS, rows);
        base = L - n;
        sinks = sink_end = skip = lo = 0;
        lim[0] = lim[1] = last = -1;
        tiles = 0;
        if (r0 >= rows || L == 0) return;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int g0 = r0 + g * QT;
            if (g0 < r_end) lim[g] = WINDOW ? base + (min(g0 + QT, r_end) - 1) / p.gh : L - 1;
        }
        last = max(lim[0], lim[1]);
        if constexpr (WINDOW) {
            lo = max(0, base + r0 / p.gh - p.mask.window + 1);   // the first row's window
            sinks = min(p.mask.sinks, last + 1);
            const int units = (sinks + (1 << p.unit_shift) - 1) >> p.unit_shift;
            sink_end = units << p.unit_shift;
            skip = max(0, (lo >> p.unit_shift) - units) << p.unit_shift;
            last -= skip;
            lo -= skip;
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if (lim[g] >= 0) lim[g] -= skip;    // (no position before the window's start)
        }
        tiles = last / BN + 1;
    }
};

// What the roles need of a block.
struct Info {
    int blk;                  // -1: no more
    int s, h, part;
    int q0, n, base;
    int r0, r_end;
    int i0, rem0;             // r0 = i0 * gh + rem0
    int lim[2], nt[2];        // per query tile: last virtual position, tiles of this part
    int last, sinks, sink_end, skip, lo;
    int tile0, tiles, n_parts;
    // context token of virtual token x (trees: itself, sink_end and skip are 0)
    __device__ __forceinline__ int token(int x) const { return x >= sink_end ? x + skip : x; }
    // some row of the block sees virtual token x (which is not past the last)
    __device__ __forceinline__ bool seen(int x) const { return x < sinks || x >= lo; }
};

// What a softmax thread keeps of it, for its query tile.
struct Rows {
    int blk, h, part, q0, n, base, r0, r_end, i0, rem0, lim, nt, sinks, skip, tile0, n_parts;
};

struct Bars {
    unsigned long long k_full[4];
    unsigned long long v_full[4];
    unsigned long long k_empty[4];
    unsigned long long v_empty[4];
    unsigned long long s_full[2];
    unsigned long long s_free[2];
    unsigned long long p_full[2];
    unsigned long long o_done[2];
    unsigned long long q_full[2];
    unsigned long long v_landed;     // a V tile with rows to clear, for its loaders
    unsigned long long ml_full[2];     // DUAL: a group's maxima and sums are there
    unsigned long long o_read[2];      // DUAL: a group has read both products
    unsigned long long mma_done[2];
    unsigned long long info_full[kInfos];
    unsigned long long info_empty[kInfos];
    uint32_t tmem_base;
};

template <int D, bool Q8, bool SPLIT, int MASK, bool DUAL>
__global__ void __launch_bounds__(NTHREADS, 1)
    prompt_masked_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const Params p) {
    using C = Cfg<D, Q8, DUAL>;
    constexpr bool WINDOW = MASK == kMaskWindow, TREE = MASK == kMaskTree;
    constexpr int BN = C::BN;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    __shared__ Info infos[kInfos];
    __shared__ uint8_t order[TREE ? kOrderSeqs : 1];         // sequences, the longest first
    static_assert(C::SMEM + sizeof(Bars) + sizeof(infos) + kOrderSeqs + 16 <= 227 * 1024, "shared memory");
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int warp = (int)threadIdx.x / 32;
    const int lane = (int)threadIdx.x % 32;
    auto bar = [](unsigned long long &x) { return smem_addr(&x); };
    // Every wait has the launch's limit: most last a tile, but warp 14's for a free
    // description a block, and those of a softmax group without tiles in some blocks
    // (their rows fit one query tile; the group goes on, up to kInfos blocks ahead)
    // as long as the other takes for them.  (wait_one: by one thread.)
    auto wait = [&](uint32_t b, uint32_t parity) { return wait_lanes(b, parity, p.status, p.wait_ns); };
    auto wait_one = [&](uint32_t b, uint32_t parity) { return mbar_wait(b, parity, p.status, 0, p.wait_ns); };

    // ---------------------------------------------------------------- setup
    const bool ordered = TREE && p.n_seqs > 1 && p.n_seqs <= kOrderSeqs && (p.max_blocks << p.block_shift) >= kOrderContext;
    if (ordered) {
        int *len_of = reinterpret_cast<int *>(sm + C::OFF_OUT);
        const int u = (int)threadIdx.x;
        const int mine = u < p.n_seqs ? p.lens[u] : 0;
        if (u < p.n_seqs) len_of[u] = mine;
        __syncthreads();
        if (u < p.n_seqs) {
            int rank = 0;
            for (int v = 0; v < p.n_seqs; ++v) rank += len_of[v] > mine || (len_of[v] == mine && v < u);
            order[rank] = (uint8_t)u;
        }
    }
    if (warp == MMA_S_WARP) {
        if (lane == 0) {
            for (int k = 0; k < NS; ++k) {
                // two loader warps arrive on each full barrier
                mbar_init(bar(bars.k_full[k]), !Q8 && p.block_size >= 16 ? 2u : 64u);
                mbar_init(bar(bars.v_full[k]), !Q8 && p.block_size >= 16 ? 2u : 64u);
                mbar_init(bar(bars.k_empty[k]), 1);
                mbar_init(bar(bars.v_empty[k]), 1);
            }
            for (int u = 0; u < 2; ++u) {
                mbar_init(bar(bars.s_full[u]), 1);
                mbar_init(bar(bars.s_free[u]), 128);
                mbar_init(bar(bars.p_full[u]), 128);
                mbar_init(bar(bars.o_done[u]), 1);
                mbar_init(bar(bars.mma_done[u]), 1);
                mbar_init(bar(bars.q_full[u]), 128);
                mbar_init(bar(bars.ml_full[u]), 128);
                mbar_init(bar(bars.o_read[u]), 128);
            }
            mbar_init(bar(bars.v_landed), 2);
            for (int k = 0; k < kInfos; ++k) {
                mbar_init(bar(bars.info_full[k]), 1);
                mbar_init(bar(bars.info_empty[k]), SOFTMAX_WARPS + 4 + 2);
            }
            mbar_init_fence();
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&bars.tmem_base)),
                     "n"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = bars.tmem_base;

    const uint32_t s_k = smem_addr(sm + C::OFF_K);
    const uint32_t s_v = smem_addr(sm + C::OFF_V);
    // The k-th block; false: a wait ran out.  (take_one: by one thread of the warp.)
    auto take = [&](unsigned k, Info &f) {
        const unsigned slot = k % kInfos;
        if (!wait(bar(bars.info_full[slot]), (k / kInfos) & 1)) return false;
        f = infos[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.info_empty[slot]));
        return true;
    };
    auto take_one = [&](unsigned k, Info &f) {
        const unsigned slot = k % kInfos;
        if (!wait_one(bar(bars.info_full[slot]), (k / kInfos) & 1)) return false;
        f = infos[slot];
        mbar_arrive(bar(bars.info_empty[slot]));
        return f.blk >= 0;
    };

    // (setmaxnreg right at the branch: with code of both kinds of warps after it
    // the softmax kept to 128 registers and spilled)
    if (warp < SOFTMAX_WARPS) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<D>::SOFTMAX));
        // ---------------------------------------------------------- softmax
        const int g = warp / 4;
        const int t = (int)threadIdx.x % 128;                  // row of the tile = tensor-memory lane
        const uint32_t lane_off = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + (uint32_t)(g * BN);
        const uint32_t t_o = tmem + lane_off + (uint32_t)(C::COL_O + g * D);
        const uint32_t t_p = tmem + lane_off + (uint32_t)(C::COL_P + g * (BN / 2));
        const uint32_t stage = smem_addr(sm + C::OFF_OUT) + warp * C::OUT_BYTES;
        const float sl = p.scale_log2;
        const int row0_g = DUAL ? 0 : g * QT;                  // of the group's query tile in the block
        float2 *ml = reinterpret_cast<float2 *>(sm + C::OFF_ML);   // DUAL: [group][row]
        unsigned done_other = 0;                               // DUAL: tiles of the other group so far
        unsigned done = 0;                                     // tiles of this query tile so far
        bool ok = true;
        Rows f;
        int nt_other = 0;
        auto take_rows = [&](unsigned k) {
            const unsigned slot = k % kInfos;
            if (!wait(bar(bars.info_full[slot]), (k / kInfos) & 1)) return false;
            const Info &in = infos[slot];
            f = Rows{in.blk, in.h, in.part, in.q0, in.n, in.base, in.r0, in.r_end, in.i0, in.rem0, in.lim[g], in.nt[g],
                     in.sinks, in.skip, in.tile0, in.n_parts};
            nt_other = in.nt[g ^ 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bars.info_empty[slot]));
            return true;
        };
        // The warp's query rows in block f (zeros past the last), 16 bytes each and
        // neighbouring lanes neighbouring chunks: on their way, then there.
        auto fetch_rows = [&]() {
            if (f.blk < 0 || f.nt == 0 || (DUAL && g)) return;   // (DUAL: the first group's rows serve both)
            constexpr int CH = D / 8;
            const int u = (warp % 4) * 32 + lane / CH, c = lane % CH;   // of the tile: this lane's first row, chunk
            const int d0 = f.rem0 + row0_g + u;
            const int left = f.r_end - f.r0 - row0_g - u;
            const __half *src = p.q + ((size_t)(f.q0 + f.i0) * p.n_q_heads + (size_t)f.h * p.gh) * D + c * 8;
            const int apart = (p.n_q_heads - p.gh) * D;        // from a token's last row to the next one's first, less a row
            const uint32_t dst = smem_addr(sm) + g * C::Q_BYTES;
#pragma unroll
            for (int it = 0; it < CH; ++it) {
                const int d = it * (32 / CH);
                const int i = ((d0 + d) * p.gh_magic) >> 16;   // tokens from i0 on
                cp_async16_zfill(dst + swz(u + d, c, QT), src + (d < left ? i * apart + (d0 + d) * D : 0), d < left ? 16u : 0u);
            }
        };
        auto rows_there = [&]() {
            if (f.blk < 0 || f.nt == 0 || (DUAL && g)) return;
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (C::Q0_TMEM && g == 0) {
                __syncwarp();
                // this thread's row, which the warp has copied, into tensor memory
#pragma unroll
                for (int c0 = 0; c0 < D / 8; c0 += 4) {
                    uint32_t x[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x[4 * c]), "=r"(x[4 * c + 1]), "=r"(x[4 * c + 2]), "=r"(x[4 * c + 3])
                                     : "r"(smem_addr(sm) + swz(t, c0 + c, QT)));
                    tmem_st16(tmem + lane_off + (uint32_t)(C::COL_Q + c0 * 4), x);
                }
                tmem_st_wait();
                tc_before_sync();
            } else {
                fence_proxy_async_shared();
            }
            mbar_arrive(bar(bars.q_full[g]));
        };
        ok = take_rows(0);
        if (ok) {
            fetch_rows();
            rows_there();
        }
        for (unsigned block = 1; ok && f.blk >= 0; ++block) {
            const size_t part_row = SPLIT ? ((size_t)f.blk * p.splits + f.part) * ROWS : 0;
            const int nt = f.nt, i0 = f.i0, rem0 = f.rem0;
            const bool valid = f.r0 + row0_g + t < f.r_end;
            const int mine = valid ? i0 + (((rem0 + row0_g + t) * p.gh_magic) >> 16) : 0;   // this row's new token
            // from the CTA's first tile on: the last virtual position that the row
            // sees, the sinks' end, the first draft
            const int from = f.tile0 * BN;
            const int lim = (WINDOW && valid ? f.base + mine - f.skip : f.lim) - from;
            const int sinks = f.sinks - from;
            const int draft0 = f.base - from;
            // the lowest n bits
            auto below = [](int n) -> uint64_t { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull); };
            // TREE: which of drafts d .. d + 63 this row sees, d > -BN (what lies before draft 0: all)
            const uint64_t *words = TREE ? p.mask.tree + (size_t)(f.q0 + mine) * p.mask.tree_words : nullptr;
            const int drafts = valid ? f.n : 0;
            auto sees_drafts = [&](int d) -> uint64_t {
                if (d <= -64) return ~0ull;
                auto word = [&](int k) -> uint64_t {           // of the drafts' bits
                    const int left = drafts - 64 * k;
                    return left <= 0 ? 0ull : words[k] & below(left);
                };
                if (d < 0) return (word(0) << -d) | below(-d);
                const int k = d / 64, sh = d % 64;
                return sh ? (word(k) >> sh) | (word(k + 1) << (64 - sh)) : word(k);
            };
            float m = -INFINITY;                               // reference maximum, log2 units
            float l = 0.0f;                                    // sum of the weights
            for (int j = 0; j < nt; ++j, ++done) {
                if (!wait(bar(bars.s_full[g]), done & 1)) {
                    ok = false;
                    break;
                }
                tc_after_sync();
                uint32_t x[BN];                                // raw scores (fp32 bits)
#pragma unroll
                for (int q = 0; q < BN / 32; ++q) tmem_ld32(t_s + q * 32, x + q * 32);
                tmem_ld_wait();
                tc_before_sync();
                mbar_arrive(bar(bars.s_free[g]));              // the MMA warp may overwrite S

                // What the row does not see: -inf.  A bit per column says what it
                // sees (two compares and a select per column took longer).
                const int x0 = (DUAL ? 2 * j + g : j) * BN;
                const int cl = lim - x0, cw = cl - p.mask.window + 1, cs = sinks - x0;   // WINDOW
                if (TREE ? x0 + BN > draft0 : cl < BN - 1 || (cw > 0 && cs < cw && cs < BN)) {
#pragma unroll
                    for (int q = 0; q < BN / 64; ++q) {
                        uint64_t seen;
                        if constexpr (TREE) seen = sees_drafts(x0 + 64 * q - draft0);
                        else seen = below(cl + 1 - 64 * q) & (~below(cw - 64 * q) | below(cs - 64 * q));
                        const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!(((c < 32 ? lo : hi) >> (c & 31)) & 1u)) x[64 * q + c] = 0xff800000u;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < BN; c += 8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = max3(mx[e], __uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]));
                }
                const float mt = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * sl;   // scale > 0
                float f = 1.0f;
                const bool resc = mt > m + kRescaleLog2;
                if (resc) {
                    f = ex2(m - mt);                           // m = -inf gives 0
                    m = mt;
                    l *= f;
                }
                // weights 2^(s sl - m) (nothing seen so far: all 0); their sum two at a time
                const float nm = m == -INFINITY ? 0.0f : -m;
                uint64_t ls[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
                uint32_t pk[BN / 2];
#pragma unroll
                for (int c = 0; c < BN / 2; ++c) {
                    const float w0 = ex2(fmaf(__uint_as_float(x[2 * c]), sl, nm));
                    const float w1 = ex2(fmaf(__uint_as_float(x[2 * c + 1]), sl, nm));
                    ls[c & 1] = f2_add(ls[c & 1], f2_pack(w0, w1));
                    pk[c] = pack_half2(w0, w1);
                }
                {
                    float a0, a1, b0, b1;
                    f2_unpack(ls[0], a0, a1);
                    f2_unpack(ls[1], b0, b1);
                    l += (a0 + a1) + (b0 + b1);
                }

                // DUAL: the other group has read the last block's O
                if (DUAL && j == 0 && block > 1 && !wait(bar(bars.o_read[g ^ 1]), block & 1)) {
                    ok = false;
                    break;
                }
                // the previous product has finished reading P and adding to O
                if (j > 0) {
                    if (!wait(bar(bars.o_done[g]), (done - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_after_sync();
                    if (__any_sync(FULL, resc)) {
                        // rescale O (lanes without a new maximum scale by 1)
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + c0, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(t_o + c0, o);
                        }
                        tmem_st_wait();
                    }
                }
                // P row t into tensor memory
#pragma unroll
                for (int q = 0; q < BN / 64; ++q) tmem_st32(t_p + q * 32, pk + q * 32);
                tmem_st_wait();
                tc_before_sync();
                mbar_arrive(bar(bars.p_full[g]));
            }
            if (!ok) break;
            // On to the next block: the scores of this tile are all done, so its
            // query rows can take the place of this block's while the last
            // product and the output go on.
            const int left = f.r_end - f.r0, n_parts = f.n_parts;
            const size_t row0 = ((size_t)(f.q0 + i0) * p.n_q_heads + (size_t)f.h * p.gh) * D;   // of token i0
            const int other = nt_other;
            if (DUAL) {
                // the second group's scores, over the same query rows, are done too
                // (no further ones come before the next rows); the other group has
                // read what this one left for the last block (above, with tiles)
                done_other += other;
                if (g == 0 && other > 0 && !wait(bar(bars.s_full[g ^ 1]), (done_other - 1) & 1)) break;
                if (nt == 0 && block > 1 && !wait(bar(bars.o_read[g ^ 1]), block & 1)) break;
                ml[g * QT + t] = make_float2(m, l);
                mbar_arrive(bar(bars.ml_full[g]));
            }
            ok = take_rows(block);
            if (!ok) break;
            fetch_rows();
            if (!DUAL && nt == 0) {
                rows_there();
                continue;
            }
            if (nt > 0 && !wait(bar(bars.o_done[g]), (done - 1) & 1)) break;
            float f_own = 1.0f, f_other = 0.0f;                // DUAL: factors that join the groups
            if (DUAL) {
                if ((other > 0 && !wait(bar(bars.o_done[g ^ 1]), (done_other - 1) & 1)) ||
                    !wait(bar(bars.ml_full[g ^ 1]), (block - 1) & 1))
                    break;
                const float2 o = ml[(g ^ 1) * QT + t];
                const float top = fmaxf(m, o.x);
                if (top > -INFINITY) {
                    f_own = ex2(m - top);
                    f_other = ex2(o.x - top);
                }
                m = top;
                l = l * f_own + o.y * f_other;
            }
            tc_after_sync();
            const bool whole = !SPLIT || n_parts == 1;         // else a part: unscaled, fp32
            const float inv = !whole ? 1.0f : (TREE && l == 0.0f ? 0.0f : 1.0f / l);   // (a draft may see nothing)
            if (!whole && !(DUAL && g)) p.part_ml[part_row + row0_g + t] = make_float2(m, l);
            // The warp's 32 rows, up to 128 bytes of each at a time, through shared
            // memory: stored by rows straight from tensor memory, 16 bytes per
            // lane and row, the output took 5,000 cycles.  (DUAL: each group half of
            // the dims, from both products.)
            const int t0 = (warp % 4) * 32;
            const uint32_t o_0 = tmem + lane_off + (uint32_t)C::COL_O;
            auto store = [&](auto f32_c) {
                constexpr bool F32 = decltype(f32_c)::value;
                constexpr int DIMS = DUAL ? D / 2 : D;         // of this group
                constexpr int DP = F32 ? 32 : (DIMS < 64 ? DIMS : 64);   // at a time
                constexpr int CK = DP * (F32 ? 4 : 2) / 16;    // chunks of them
                const int first = DUAL ? g * DIMS : 0;
#pragma unroll 1
                for (int c0 = 0; c0 < DIMS; c0 += DP) {
#pragma unroll
                    for (int half = 0; half < DP / 32; ++half) {
                        uint32_t o[32];
                        float by = inv;
                        if constexpr (DUAL) {
                            const int at = first + c0 + half * 32;
                            const float f0 = (g ? f_other : f_own) * inv, f1 = (g ? f_own : f_other) * inv;
                            uint32_t u[32];
                            tmem_ld32(o_0 + at, o);
                            if (g ? nt > 0 : other > 0) {      // (the second group has tiles)
                                tmem_ld32(o_0 + D + at, u);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(fmaf(__uint_as_float(u[e]), f1, __uint_as_float(o[e]) * f0));
                                by = 1.0f;
                            } else {
                                tmem_ld_wait();
                                by = f0;
                            }
                        } else {
                            tmem_ld32(t_o + c0 + half * 32, o);
                            tmem_ld_wait();
                        }
#pragma unroll
                        for (int e = 0; e < (F32 ? 8 : 4); ++e) {
                            uint32_t v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if constexpr (F32) v[k] = __float_as_uint(__uint_as_float(o[4 * e + k]) * by);
                                else v[k] = pack_half2(__uint_as_float(o[8 * e + 2 * k]) * by,
                                                       __uint_as_float(o[8 * e + 2 * k + 1]) * by);
                            }
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + swz(lane, half * 4 + e, 32)),
                                         "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                         : "memory");
                        }
                    }
                    __syncwarp();
                    if (DUAL && c0 + DP == DIMS) {             // both products have been read
                        tc_before_sync();
                        mbar_arrive(bar(bars.o_read[g]));
                    }
                    if (c0 == 0) rows_there();                 // the next block's scores can begin
#pragma unroll
                    for (int it = 0; it < CK; ++it) {
                        const int row = it * (32 / CK) + lane / CK, c = lane % CK, d = row0_g + t0 + row;
                        uint4 v;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(stage + swz(row, c, 32)));
                        const int col = first + c0 + c * (F32 ? 4 : 8);
                        if (SPLIT && !whole) {
                            if (F32 && d < left) *reinterpret_cast<uint4 *>(p.part_o + (part_row + d) * D + col) = v;
                        } else if (d < left) {
                            const int i = ((rem0 + d) * p.gh_magic) >> 16;   // tokens from i0 on
                            const size_t at = row0 + ((size_t)i * p.n_q_heads + (rem0 + d - i * p.gh)) * D + col;
                            if constexpr (F32) *reinterpret_cast<uint4 *>(static_cast<float *>(p.out) + at) = v;
                            else *reinterpret_cast<uint4 *>(static_cast<__half *>(p.out) + at) = v;
                        }
                    }
                    __syncwarp();
                }
            };
            if (p.out_f32 || !whole) store(std::true_type());
            else store(std::false_type());
            tc_before_sync();                                  // O has been read: the next block's P says so
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<D>::OTHER));
    if (warp < MMA_S_WARP) {
        // ---------------------------------------------------------- loaders
        const bool is_v = warp >= LOAD_WARP0 + 2;
        const int li = (warp - LOAD_WARP0) & 1;
        const CUtensorMap *map = is_v ? &tmv : &tmk;
        unsigned long long *full = is_v ? bars.v_full : bars.k_full;
        unsigned long long *empty = is_v ? bars.v_empty : bars.k_empty;
        const uint32_t s_base = is_v ? s_v : s_k;
        const int B = p.block_size;
        const int32_t *bt_row = nullptr;
        int h = 0, last = -1;                                  // kv-head; the CTA's last virtual token of the block
        unsigned issued = 0;                                   // tiles so far
        // the stage of the next tile, once the MMAs over what it holds are done
        auto stage_free = [&]() {
            return issued < (unsigned)NS || wait(bar(empty[issued % NS]), (issued / NS - 1) & 1);
        };
        bool ok = true;
        Info f = {};
        if constexpr (!Q8) {
            prefetch_tensormap(map);
            const __half *pool_base = static_cast<const __half *>(is_v ? p.v_pool : p.k_pool);
            const int box = 1 << p.unit_shift;
            unsigned landed = 0;
            for (unsigned block = 0; ok && take(block, f) && f.blk >= 0; ++block) {
                bt_row = p.bt + (size_t)f.s * p.max_blocks;
                h = f.h;
                last = min(f.last, (f.tile0 + f.tiles) * BN - 1);
                // Block size 16 and up: block id of box `lane` of a tile (boxes past
                // the last token are not loaded), read two tiles ahead of its use
                // and range-checked only when used.
                auto n_boxes = [&](int j) { return min(BN >> p.unit_shift, ((last - (f.tile0 + j) * BN) >> p.unit_shift) + 1); };
                auto box_id = [&](int j) {
                    return B >= 16 && j < f.tiles && lane < n_boxes(j)
                               ? bt_row[f.token((f.tile0 + j) * BN + lane * box) >> p.block_shift]
                               : 0;
                };
                int id0 = box_id(0), id1 = box_id(1);
                for (int j = 0; j < f.tiles; ++j, ++issued) {
                    int id = id0;
                    id0 = id1;
                    id1 = box_id(j + 2);
                    const int st = issued % NS;
                    const uint32_t dst = s_base + st * C::KV_BYTES;
                    const int x0 = (f.tile0 + j) * BN;
                    if (!stage_free()) {
                        ok = false;
                        break;
                    }
                    if (B >= 16) {
                        const int nb = n_boxes(j);
                        const bool mine = lane < nb && (lane & 1) == li;   // every other box
                        if (mine && (unsigned)id >= (unsigned)p.n_blocks) {
                            atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                            id = 0;
                        }
                        // Rows of V past the last token, and others that no row sees,
                        // become zeros (a zero weight times a non-finite value would not
                        // vanish): such a tile lands on a barrier of its own first.
                        const int rows = last - x0 + 1;
                        const bool ragged = is_v && (rows < BN || (WINDOW && f.sinks < f.lo && f.sinks < x0 + BN && f.lo > x0));
                        const uint32_t on = bar(ragged ? bars.v_landed : full[st]);
                        if (lane == 0) mbar_arrive_expect_tx(on, (uint32_t)((nb + 1 - li) / 2) * box * D * 2);
                        __syncwarp();
                        if (mine) {
                            const int row = (int)(p.layer_row0 + (long long)id * B + (f.token(x0 + lane * box) & (B - 1)));
#pragma unroll
                            for (int hf = 0; hf < C::HALVES; ++hf)
                                tma_load_4d_plain(dst + (uint32_t)(hf * BN + lane * box) * 128u, map, 0, row, hf, h, on);
                        }
                        if (ragged) {
                            if (!wait(on, landed & 1)) {
                                ok = false;
                                break;
                            }
                            ++landed;
                            const int from = WINDOW ? 0 : rows;
                            for (int e = lane; e < (BN - from) * 4 * C::HALVES; e += 32) {
                                const int row = from + e / (4 * C::HALVES), rest = e % (4 * C::HALVES) * 2 + li;
                                if (WINDOW && row < rows && f.seen(x0 + row)) continue;
                                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 dst + ((rest / 8) * BN + row) * 128 + (rest % 8) * 16), "r"(0u)
                                             : "memory");
                            }
                            fence_proxy_async_shared();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(full[st]));
                        }
                    } else {
                        // one token per page: 16-byte cp.async per chunk into its
                        // swizzled place, then a proxy fence before the arrival
                        for (int tk = lane + 32 * li; tk < BN; tk += 64) {
                            if (x0 + tk > last) {              // V: zeros, as above
                                if (!is_v) break;
#pragma unroll
                                for (int c = 0; c < D / 8; ++c)
                                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + swz(tk, c, BN)), "r"(0u)
                                                 : "memory");
                                continue;
                            }
                            int bid = bt_row[f.token(x0 + tk)];
                            if ((unsigned)bid >= (unsigned)p.n_blocks) {
                                atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                                bid = 0;
                            }
                            const __half *src = pool_base + ((size_t)(p.layer_row0 + bid) * p.n_kv_heads + h) * D;
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) cp_async16_cg(dst + swz(tk, c, BN), src + c * 8);
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        fence_proxy_async_shared();
                        mbar_arrive(bar(full[st]));
                    }
                }
            }
            // copies still in flight (only after a wait ran out) land before the CTA
            // exits (those of a last V tile have been waited for)
            if (B >= 16) {
                for (unsigned k = issued < (unsigned)NS ? 0 : issued - NS; k < issued; ++k)
                    wait(bar(full[k % NS]), (k / NS) & 1);
            }
        } else {
            // The tile's 512 16-byte chunks of codes are dealt to the 64 lanes of
            // the tensor's two warps: a lane copies (into a stage of codes) the
            // chunks that it widens itself; chunk i is chunk c0 of token 2 TPI i + TPI
            // li + tk (eight neighbouring lanes store to one half of two tokens'
            // rows: of both halves of one they met in the banks, 57 us for 54, 16
            // blocks of 20 drafts x 4 heads over 4,096 tokens).  Lane l looks up the block ids (one tile ahead of their
            // copy) and copies the scales of the warp's tokens l, l + 32 (in order).
            constexpr int CPR = D / 16;                        // chunks of a row of codes
            constexpr int TPI = 32 / CPR;                      // tokens of a warp per chunk index
            constexpr int TW = BN / 2;                         // tokens of a warp
            constexpr int IDS = TW / 32;
            auto tile_token = [&](int lt) { return lt / TPI * (2 * TPI) + li * TPI + lt % TPI; };
            const uint32_t raw = smem_addr(sm + C::OFF_RAW) + (is_v ? C::RAW * C::RAW_BYTES : 0);
            const float *scale_base = is_v ? p.v_scale : p.k_scale;
            int q_id[IDS];                                     // raw ids of the next tile to copy (any number; -2 where no row sees the token)
            auto look_up = [&](int j) {
#pragma unroll
                for (int k = 0; k < IDS; ++k) {
                    const int x = (f.tile0 + j) * BN + tile_token(lane + 32 * k);
                    q_id[k] = x <= last && (!WINDOW || f.seen(x)) ? bt_row[f.token(x) >> p.block_shift] : -2;
                }
            };
            // this lane's chunk 0 in a stage of codes, in the pool and in a swizzled
            // stage; chunk i is 2 TPI tokens further (t mod 8, the swizzle, stays)
            const int tk = D == 64 ? lane / 4 : (lane >> 2 & 1) | (lane >> 4) << 1;
            const int t0 = li * TPI + tk, c0 = D == 64 ? lane % 4 : (lane & 3) | (lane >> 3 & 1) << 2;
            const uint32_t raw_at = (uint32_t)(li * 32 + lane) * 16;
            const uint32_t row_bytes = (uint32_t)p.n_kv_heads * D;
            const uint8_t *codes = nullptr;
            const uint32_t wide_at[2] = {swz(t0, 2 * c0, BN), swz(t0, 2 * c0 + 1, BN)};
            auto copy = [&](int j) {                           // tile j into stage of codes j mod RAW
                const uint32_t dst = raw + (uint32_t)(j % C::RAW) * C::RAW_BYTES;
                if (j < f.tiles) {
                    int row[IDS];
                    bool whole = true;
#pragma unroll
                    for (int k = 0; k < IDS; ++k) {
                        const int id = q_id[k], lt = lane + 32 * k;
                        const bool good = (unsigned)id < (unsigned)p.n_blocks;
                        const int x = (f.tile0 + j) * BN + tile_token(lt);
                        if (!good && x <= last && (!WINDOW || f.seen(x))) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                        row[k] = good ? (int)p.layer_row0 + (id << p.block_shift) + (f.token(x) & (B - 1)) : -1;
                        whole = whole && good;
                        cp_async4_zfill(dst + BN * D + (li * TW + lt) * 4,
                                        scale_base + (good ? (size_t)(unsigned)((int)p.layer_page0 + id) * p.n_kv_heads + h : 0),
                                        good ? 4u : 0u);
                    }
                    if (__all_sync(FULL, whole)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r8 = __shfl_sync(FULL, row[i * TPI / 32], i * TPI % 32 + tk);
                            cp_async16_cg(dst + raw_at + i * 1024, codes + (size_t)(unsigned)r8 * row_bytes);
                        }
                    } else {                                   // the end, or bad ids: zeros
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r8 = __shfl_sync(FULL, row[i * TPI / 32], i * TPI % 32 + tk);
                            cp_async16_zfill(dst + raw_at + i * 1024,
                                             codes + (r8 < 0 ? 0 : (size_t)(unsigned)r8 * row_bytes), r8 < 0 ? 0u : 16u);
                        }
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (j + 1 < f.tiles) look_up(j + 1);
            };
            // tile j from its stage of codes into the next swizzled stage; false if a wait ran out
            auto widen = [&](int j) -> bool {
                const uint32_t src = raw + (uint32_t)(j % C::RAW) * C::RAW_BYTES;
                const int st = issued % NS;
                const uint32_t dst = s_base + st * C::KV_BYTES;
                if (!stage_free()) return false;
                constexpr int AT_ONCE = D == 64 ? 2 : 8;
#pragma unroll
                for (int i0 = 0; i0 < 8; i0 += AT_ONCE) {
                    uint4 c[AT_ONCE];
                    float f[AT_ONCE];
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i) {
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(c[i].x), "=r"(c[i].y), "=r"(c[i].z), "=r"(c[i].w)
                                     : "r"(src + raw_at + (i0 + i) * 1024));
                        asm volatile("ld.shared.f32 %0, [%1];"
                                     : "=f"(f[i])
                                     : "r"(src + BN * D + (li * TW + (i0 + i) * TPI + tk) * 4));
                    }
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i) {
                        const __half2 f2 = __float2half2_rn(f[i]);
                        const uint32_t in[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __half2 v = __hmul2(widen_e4m3(in[2 * k + e / 2] >> (16 * (e & 1))), f2);
                                x[e] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + wide_at[k] + (i0 + i) * 2 * TPI * 128),
                                         "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                                         : "memory");
                        }
                    }
                }
                fence_proxy_async_shared();
                mbar_arrive(bar(full[st]));
                ++issued;
                return true;
            };
            for (unsigned block = 0; ok && take(block, f) && f.blk >= 0; ++block) {
                bt_row = p.bt + (size_t)f.s * p.max_blocks;
                h = f.h;
                last = min(f.last, (f.tile0 + f.tiles) * BN - 1);
                codes = static_cast<const uint8_t *>(is_v ? p.v_pool : p.k_pool) + h * D + c0 * 16;
                look_up(0);
                __syncwarp();                                  // the stages of codes have been read
#pragma unroll 1
                for (int j = 0; j < C::RAW - 1; ++j) copy(j);
                for (int j = 0; ok && j < f.tiles; ++j) {
                    __syncwarp();                              // the stage of codes of tile j - 1 has been read
                    copy(j + C::RAW - 1);
                    asm volatile("cp.async.wait_group %0;" ::"n"(C::RAW - 1) : "memory");
                    __syncwarp();
                    ok = widen(j);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp == MMA_S_WARP) {
        // ------------------------------------------------- MMA: S = Q K^T
        constexpr uint32_t ID_S = idesc_f16(QT, BN, false);
        if (elect_one()) {
            const uint64_t dq = sdesc(smem_addr(sm)), dk = sdesc(s_k);
            bool ok = true;
            int st = 0, phase = 0;
            unsigned done[2] = {0, 0}, blocks[2] = {0, 0};
            Info f;
            for (unsigned block = 0; ok && take_one(block, f); ++block) {
                for (int j = 0; ok && j < f.tiles; ++j) {
                    if (!wait_one(bar(bars.k_full[st]), phase)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (DUAL ? (j & 1) != g : j >= f.nt[g]) continue;
                        if (j == 0 && !wait_one(bar(bars.q_full[g]), blocks[g]++ & 1)) {
                            ok = false;
                            break;
                        }
                        // S of this query tile has been read (its previous tile)
                        if (done[g] > 0 && !wait_one(bar(bars.s_free[g]), (done[g] - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        ++done[g];
                        tc_after_sync();
                        const uint64_t a = dq + (DUAL ? 0 : g) * (C::Q_BYTES / 16), kd = dk + st * (C::KV_BYTES / 16);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t k16 = kd + (kk / 4) * (BN * 128 / 16) + (kk % 4) * 2;
                            if (C::Q0_TMEM && (DUAL || g == 0)) umma_ts(tmem + g * BN, tmem + C::COL_Q + kk * 8, k16, ID_S, kk > 0);
                            else umma(tmem + g * BN, a + (kk / 4) * (QT * 128 / 16) + (kk % 4) * 2, k16, ID_S, kk > 0);
                        }
                        umma_commit(bar(bars.s_full[g]));
                    }
                    if (ok) umma_commit(bar(bars.k_empty[st]));
                    if (++st == NS) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            // every MMA issued has completed before tensor memory is released
            umma_commit(bar(bars.mma_done[0]));
        }
        __syncwarp();
        wait(bar(bars.mma_done[0]), 0);
    } else if (warp == MMA_PV_WARP) {
        // ------------------------------------------------ MMA: O += P V
        constexpr uint32_t ID_PV = idesc_f16(QT, D, true);
        if (elect_one()) {
            const uint64_t dv = sdesc(s_v, BN * 128);
            bool ok = true;
            int st = 0, phase = 0;
            unsigned done[2] = {0, 0};
            Info f;
            for (unsigned block = 0; ok && take_one(block, f); ++block) {
                for (int j = 0; ok && j < f.tiles; ++j) {
                    if (!wait_one(bar(bars.v_full[st]), phase)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (DUAL ? (j & 1) != g : j >= f.nt[g]) continue;
                        if (!wait_one(bar(bars.p_full[g]), done[g]++ & 1)) {
                            ok = false;
                            break;
                        }
                        tc_after_sync();
                        const uint64_t vd = dv + st * (C::KV_BYTES / 16);
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk)
                            umma_ts(tmem + C::COL_O + g * D, tmem + C::COL_P + g * (BN / 2) + kk * 8, vd + kk * (2048 / 16),
                                    ID_PV, j > (DUAL ? 1 : 0) || kk > 0);
                        umma_commit(bar(bars.o_done[g]));
                    }
                    if (ok) umma_commit(bar(bars.v_empty[st]));
                    if (++st == NS) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            umma_commit(bar(bars.mma_done[1]));
        }
        __syncwarp();
        wait(bar(bars.mma_done[1]), 0);
    } else if (warp == INFO_WARP) {
        // ----------------------------------------------- what the blocks are
        // Work w: part w mod splits of block w / splits, the longest blocks first.  Of
        // n = (rounds - 1) grid + few, the first (rounds - 1) (grid - few) go to
        // grid - few CTAs, rounds - 1 each, and the last rounds x few to `few` CTAs, to
        // and fro over either: who takes a block more takes the short ones.
        const int grid = (int)gridDim.x, rounds = (p.n_work - 1) / grid + 1, few = p.n_work - (rounds - 1) * grid;
        const bool more = (int)blockIdx.x >= grid - few;
        const int mine = more ? rounds : rounds - 1, width = more ? few : grid - few;
        const int col = more ? (int)blockIdx.x - (grid - few) : (int)blockIdx.x;
        const int first = more ? (rounds - 1) * (grid - few) : 0;
        struct Work {
            int s, h, qp, part, blk;                           // blk < 0: none
        };
        auto work_at = [&](int round) {
            Work w;
            w.blk = -1;
            w.s = w.h = w.qp = w.part = 0;
            if (round >= mine) return w;
            const int at = first + round * width + (round & 1 ? width - 1 - col : col);
            const int b = SPLIT ? at / p.splits : at;
            w.part = SPLIT ? at - b * p.splits : 0;
            if (TREE) {                                        // by sequences
                const int per = p.n_kv_heads * p.n_qp, rank = b / per, rest = b - rank * per;
                w.s = ordered ? order[rank] : rank;
                w.qp = rest / p.n_kv_heads;
                w.h = rest - w.qp * p.n_kv_heads;
            } else {                                           // by query rows, the last first
                const int up = b / p.n_items, item = b - up * p.n_items;
                w.qp = p.n_qp - 1 - up;
                w.s = item / p.n_kv_heads;
                w.h = item - w.s * p.n_kv_heads;
            }
            w.blk = (w.s * p.n_kv_heads + w.h) * p.n_qp + w.qp;
            return w;
        };
        const bool step = WINDOW && !p.cu_q;
        auto seq_of = [&](const Work &w) {
            Seq q;
            q.L = p.lens[w.s];
            q.q0 = step ? w.s : p.cu_q[w.s];
            q.q1 = step ? w.s + 1 : p.cu_q[w.s + 1];
            return q;
        };
        // to the roles; false: a wait ran out
        unsigned k = 0;
        auto publish = [&](const Info &f) {
            const unsigned slot = k % kInfos;
            if (k >= kInfos && !wait(bar(bars.info_empty[slot]), (k / kInfos - 1) & 1)) return false;
            if (lane == 0) {
                infos[slot] = f;
                mbar_arrive(bar(bars.info_full[slot]));
            }
            ++k;
            return true;
        };
        // 32 rounds are looked at together, a lane each: blocks without rows (with a
        // loose max_new most of them) are passed over.  The first of a (sequence,
        // kv-head) is always taken: its lengths may be bad, its output zeros.
        bool ok = true;
        for (int round0 = 0; ok && round0 < mine; round0 += 32) {
            const Work look = work_at(round0 + lane);
            const Seq look_seq = seq_of(look);
            unsigned todo = __ballot_sync(
                FULL, look.blk >= 0 && (look.qp == 0 || min(look_seq.q1 - look_seq.q0, p.max_new) * p.gh > look.qp * ROWS));
            for (; ok && todo; todo &= todo - 1) {
                const int from = __ffs(todo) - 1;
                Work w;
                Seq seq;
                w.s = __shfl_sync(FULL, look.s, from);
                w.h = __shfl_sync(FULL, look.h, from);
                w.qp = __shfl_sync(FULL, look.qp, from);
                w.part = __shfl_sync(FULL, look.part, from);
                w.blk = __shfl_sync(FULL, look.blk, from);
                seq.L = __shfl_sync(FULL, look_seq.L, from);
                seq.q0 = __shfl_sync(FULL, look_seq.q0, from);
                seq.q1 = __shfl_sync(FULL, look_seq.q1, from);
                Block<BN, MASK> b;
                Info f = {};
                bool bad;
                b.make(p, seq, w.qp, bad);
                if (bad && w.qp == 0 && w.h == 0 && w.part == 0 && lane == 0) atomicOr(p.status, PF_DEV_BAD_LENGTH);
                f.tile0 = 0;
                f.tiles = b.tiles;
                f.n_parts = 1;
                if constexpr (SPLIT) {
                    if (b.tiles > 0) {
                        const int per = part_tiles(b.tiles, p.splits);
                        f.n_parts = (b.tiles + per - 1) / per;
                        f.tile0 = w.part * per;
                        f.tiles = w.part < f.n_parts ? min(b.tiles - f.tile0, per) : 0;
                    }
                }
                if (f.tiles == 0) {
                    if (step && w.part == 0 && b.L == 0 && b.r0 < b.n * p.gh) {
                        // a decode step over an empty context: zeros
                        for (int e = lane; e < (b.r_end - b.r0) * (D / 8); e += 32) {
                            const size_t o = ((size_t)b.q0 * p.n_q_heads + (size_t)w.h * p.gh + b.r0 + e / (D / 8)) * D + e % (D / 8) * 8;
                            if (p.out_f32) {
                                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + o);
                                dst[0] = dst[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            } else {
                                *reinterpret_cast<uint4 *>(static_cast<__half *>(p.out) + o) = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    }
                    continue;
                }
                f.blk = w.blk;
                f.s = w.s, f.h = w.h, f.part = w.part;
                f.q0 = b.q0, f.n = b.n, f.base = b.base, f.r0 = b.r0, f.r_end = b.r_end;
                f.i0 = b.r0 / p.gh;
                f.rem0 = b.r0 - f.i0 * p.gh;
                f.last = b.last, f.sinks = b.sinks, f.sink_end = b.sink_end, f.skip = b.skip, f.lo = b.lo;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    f.lim[g] = b.lim[DUAL ? 0 : g];
                    f.nt[g] = DUAL ? (f.tiles + 1 - g) / 2 : b.lim[g] < 0 ? 0 : min(max(b.lim[g] / BN + 1 - f.tile0, 0), f.tiles);
                }
                ok = publish(f);
            }
        }
        if (ok) {
            Info f = {};
            f.blk = -1;                                        // no more
            publish(f);
        }
    }
    }

    tc_before_sync();
    __syncthreads();
    if (warp == MMA_S_WARP) {
        tc_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TMEM_COLS)
                     : "memory");
    }
}

// The rows of cut blocks from their parts: with M the largest reference
// maximum m_i, out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over the parts up
// to the row's last tile.  A warp per row; lane i holds part i's m and l.
constexpr int kMergeWarps = 8;
template <int D, int MASK>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_masked_kernel(const Params p) {
    constexpr int BN = Cfg<D, false, false>::BN;
    constexpr int V = D / 32;                // values of a lane
    const int blk = (int)blockIdx.x;
    const int item = blk / p.n_qp, qp = blk - item * p.n_qp;
    const int s = item / p.n_kv_heads, h = item - s * p.n_kv_heads;
    const int lane = (int)threadIdx.x % 32;
    const int d = (int)blockIdx.y * kMergeWarps + (int)threadIdx.x / 32;   // row of the block
    griddep_wait();
    const bool step = MASK == kMaskWindow && !p.cu_q;
    Seq seq;
    seq.L = p.lens[s];
    seq.q0 = step ? s : p.cu_q[s];
    seq.q1 = step ? s + 1 : p.cu_q[s + 1];
    Block<BN, MASK> b;
    bool bad;
    b.make(p, seq, qp, bad);
    const int r = b.r0 + d;
    const int per = part_tiles(b.tiles, p.splits);
    if (b.tiles <= per || r >= b.r_end) return;   // one part: written by the main kernel
    const int i = r / p.gh;
    const int parts = (MASK == kMaskWindow ? b.base + i - b.skip : b.last) / BN / per + 1;
    const size_t row = ((size_t)blk * p.splits) * ROWS + d;
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < parts) ml = p.part_ml[row + (size_t)lane * ROWS];
    float top = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
    const float w = top == -INFINITY ? 0.0f : ex2(ml.x - top);   // (a draft may see nothing)
    float l = w * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    const float *at = p.part_o + row * D + lane * V;
#pragma unroll 8
    for (int k0 = 0; k0 < parts; ++k0) {
        const float wi = __shfl_sync(FULL, w, k0);
        float x[V];
        if constexpr (V == 2) {
            const float2 v = *reinterpret_cast<const float2 *>(at + (size_t)k0 * ROWS * D);
            x[0] = v.x, x[1] = v.y;
        } else {
            const float4 v = *reinterpret_cast<const float4 *>(at + (size_t)k0 * ROWS * D);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(wi, x[k], acc[k]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const size_t out = ((size_t)(b.q0 + i) * p.n_q_heads + (size_t)h * p.gh + (r - i * p.gh)) * D + lane * V;
#pragma unroll
    for (int k = 0; k < V; k += 2) {
        if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + out + k) = make_float2(acc[k] * inv, acc[k + 1] * inv);
        else *reinterpret_cast<__half2 *>(static_cast<__half *>(p.out) + out + k) = __floats2half2_rn(acc[k] * inv, acc[k + 1] * inv);
    }
}

// Kernels of one mask (prompt_masked_<mask>.cu).
struct Kernels {
    void (*main)(CUtensorMap, CUtensorMap, Params);
    void (*merge)(Params);   // of the parts, when contexts are cut
    int smem;
};
Kernels window_kernels(int D, bool q8, bool split, bool dual);
Kernels tree_kernels(int D, bool q8, bool split, bool dual);

template <int MASK, int D, bool Q8>
Kernels kernels_of(bool split, bool dual) {
    const auto main = split ? (dual ? prompt_masked_kernel<D, Q8, true, MASK, true> : prompt_masked_kernel<D, Q8, true, MASK, false>)
                            : (dual ? prompt_masked_kernel<D, Q8, false, MASK, true> : prompt_masked_kernel<D, Q8, false, MASK, false>);
    return {main, merge_masked_kernel<D, MASK>, dual ? Cfg<D, Q8, true>::SMEM : Cfg<D, Q8, false>::SMEM};
}
template <int MASK, int D>
Kernels kernels_of(bool q8, bool split, bool dual) {
    return q8 ? kernels_of<MASK, D, true>(split, dual) : kernels_of<MASK, D, false>(split, dual);
}

}  // namespace prompt_masked
}  // namespace pkv
