// prefill_tc.cu -- prompt attention through the block tables on the
// fifth-generation tensor cores: tcgen05.mma with fp32 accumulators in
// tensor memory (pf_paged_prefill_attention calls with 128 or more query
// rows per (sequence, kv-head)); also, in instances of their own, over e4m3
// pools and without the causal limit (pf_paged_cross_attention).
//
// Sequence s has L_s tokens, the last n_s of them new (PagedAttention blog,
// "Architecture": append into the last block, then attend); the query of new
// token i sits at position p = L_s - n_s + i and attends causally to tokens
// 0 .. p.  A kv-head's query rows are its new tokens x its gh q-heads, row
// r = i * gh + g.
//
// A CTA serves 256 consecutive rows of one (sequence, kv-head) as two query
// tiles of 128 rows (the MMA's M), with sixteen warps:
//   warps 0-3 and 4-7  the softmax of query tile 0 and 1: thread t owns row t
//                      of its tile, which is lane t of tensor memory;
//   warps 8-11         the loaders, two for K and two for V: tiles of BN
//                      tokens (128 at head_dim 64, 64 at 128) through the
//                      block table into a ring of four stages in the
//                      128-byte swizzle, by TMA boxes of up to a page (block
//                      size 16 and up; each warp every other box) or 16-byte
//                      cp.async per token (block size 1);
//   warp 12            one elected thread issues the scores S_g = Q_g K_j^T (A
//                      and B in shared memory); owns the tensor memory;
//   warp 13            one elected thread issues the products O_g += P_g V_j
//                      (P in tensor memory, V in shared memory);
//   warp 14            zeroes the V rows past the last position (fp16 pools);
//                      warp 15 idles.
// The softmax warpgroups run with more registers a thread than the others
// (setmaxnreg after the setup barrier).
// The softmax threads read their row of S, apply the causal limit, keep a
// running maximum per row (raised only past 2^8, log2 domain, so O is
// rescaled rarely), add their weights to the row sum in fp32 and write them,
// rounded to fp16, back to tensor memory as P_g.  Scores and products are
// issued by separate warps so that one's waits leave the tensor pipe to the
// other; with four stages the scores of the next tiles are computed while
// the softmax threads exponentiate.
//
// Measured (GB300; 4 prompts of 2048 tokens): 12 heads x 64 46 us, 32 q-heads
// over 8 kv-heads x 128 142 us, over an e4m3 pool 145 us.  A K/V step at head_dim
// 64 takes 2,400 cycles (clock64), and no pipe is full: the exponentials of two
// query tiles are 1,024 cycles at the 32 per cycle and SM that a loop of
// ex2.approx reaches, and whole cross prompts have the issue slots 51 %, the
// tensor pipe 32 % and the MUFU pipe 34 % busy.  A step is a chain (scores,
// maximum, exponentials, P, product) in two softmax warps per scheduler, so its
// latency counts: P lives in tensor memory, the row sums are summed on the CUDA
// cores rather than by another MMA over P, and nothing else of a step may wait.
// TMA boxes issued from one warp arrive at a few hundred cycles each whatever
// their size, and the rate grows with the number of issuing warps (measured:
// 1, 2, 4 warps -> 11.8, 23.4, 44 bytes a cycle per SM on 8 KB boxes), hence
// two loader warps per tensor; 16-byte cp.async from the loader warps was
// several times slower than TMA.
//
// e4m3 pools (Q8): the loader warps bring each tile's codes into a ring of
// raw stages by 16-byte cp.async (a lane copies the chunks that it widens
// itself), widen them to fp16, multiply by the page's scale (exact but where
// the product falls below fp16's smallest normal, then off by at most 2^-25)
// and store them into the swizzled stage that the MMAs read; rows past the
// last position are zero-filled.
//
// Contexts cut over the SMs (SPLIT: few blocks, long contexts, a workspace): a
// block (sequence, kv-head, query rows) is one CTA per part of its context.  A
// part's CTA counts positions and tiles from its first token and leaves O, not
// yet divided, with each row's maximum and sum of weights in the workspace;
// merge_parts_kernel joins them.  A block whose context fills one part only
// writes its output itself.  (prompt_splits has the rule and both sides.)
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>
#include <type_traits>

#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace prefill_tc {
namespace {

constexpr int QT = 128;          // rows per query tile (the MMA's M)
constexpr int SOFTMAX_WARPS = 8;  // warpgroups 0 and 1
constexpr int LOAD_WARP0 = 8;     // warpgroup 2: K loaders (warps 8, 9), V loaders (10, 11)
constexpr int MMA_S_WARP = 12;    // warpgroup 3: issues the scores; owns the tensor memory
constexpr int MMA_PV_WARP = 13;   // issues the products
constexpr int CLEAN_WARP = 14;    // zeroes V rows past the end (warp 15 idles)
constexpr int NTHREADS = 512;
// Registers: launched at 128 a thread (512 threads, one CTA per SM); the
// loader and MMA warpgroups then give some of theirs to the softmax
// warpgroups, which at head_dim 64 hold 128 scores and their weights a row (64
// at 128: the loaders of e4m3 tiles keep more).  Each SM sub-partition holds
// one warp of every warpgroup, so the split must also fit its 16K registers.
template <int D>
struct Regs {
    static constexpr int SOFTMAX = D == 64 ? 200 : 152;
    static constexpr int OTHER = 256 - SOFTMAX;
    static_assert(SOFTMAX % 8 == 0 && 2 * 128 * (SOFTMAX + OTHER) == NTHREADS * 128, "the split is the launch's registers");
    static_assert(32 * (2 * SOFTMAX + 2 * OTHER) <= 16384, "a sub-partition's registers");
};
constexpr int kOrderSeqs = NTHREADS;   // a thread per sequence
constexpr int kOrderContext = 1024;
// Long contexts of few blocks are cut into parts of at least kMinTiles tiles,
// at most kMaxParts of them (a lane each in the merge).
constexpr int kMinTiles = 4;
constexpr int kMaxParts = 32;
constexpr int kRawStages = 3;    // e4m3: raw K/V stages
constexpr int TMEM_COLS = 512;
constexpr float kRescaleLog2 = 8.0f;
constexpr unsigned FULL = 0xffffffffu;

template <int D, bool Q8>
struct Cfg {
    static constexpr int NS = Q8 ? 3 : 4;               // K/V stages
    static constexpr int BN = D == 64 ? 128 : 64;       // tokens per K/V tile (the scores' N)
    static constexpr int HALVES = D / 64;               // 64-element halves of a row
    static constexpr int Q_BYTES = QT * D * 2;          // one query tile
    static constexpr int KV_BYTES = BN * D * 2;         // one K or V tile
    static constexpr int OFF_K = 2 * Q_BYTES;
    static constexpr int OFF_V = OFF_K + NS * KV_BYTES;
    static constexpr int OFF_RAW = OFF_V + NS * KV_BYTES;
    // e4m3: codes of a K or V tile, then the scales of its tokens
    static constexpr int RAW_BYTES = Q8 ? BN * D + BN * 4 : 0;
    static constexpr int DATA = OFF_RAW + 2 * kRawStages * RAW_BYTES;
    static constexpr int SMEM = DATA + 1024;            // slack to align the base to 1024 bytes
    // tensor memory (fp32 columns): S of query tile g at g BN, O of tile g at
    // 2 BN + g D, and the fp16 weights P of tile g, two per column (token 2c
    // in the low half of column c), at 2 BN + 2 D + g BN / 2
    static constexpr int COL_O = 2 * BN;
    static constexpr int COL_P = COL_O + 2 * D;
    static_assert(COL_P + BN <= TMEM_COLS, "tensor memory columns");
    static_assert(SMEM <= 227 * 1024, "shared memory");
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
    const int32_t *cu_q;
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
    int box_rows;     // rows of one TMA box (block size 16 and up)
    int n_seqs;
    int n_items;      // sequences x kv-heads
    int n_qp;         // 256-row tiles of the longest (sequence, kv-head)
    long long layer_row0;
    long long layer_page0;   // layer * n_blocks
    int out_f32;
    float scale_log2;
    // contexts cut: the parts of block (item, qp), part after part
    int splits;       // parts at most
    float2 *part_ml;  // [block][part][2 QT]: a row's reference maximum (log2) and sum of weights
    float *part_o;    // [block][part][2 QT][D]: its sum of weighted values
};

// Tiles of a part when a block's n tiles are cut into at most `splits`.
__device__ __forceinline__ int part_tiles(int n, int splits) { return max(kMinTiles, (n + splits - 1) / splits); }

struct Bars {
    unsigned long long k_full[4];
    unsigned long long v_full[4];
    unsigned long long k_empty[4];
    unsigned long long v_empty[4];
    unsigned long long s_full[2];
    unsigned long long s_free[2];
    unsigned long long p_full[2];
    unsigned long long o_done[2];
    unsigned long long mma_done[2];
    unsigned long long v_last;       // the last V tile has landed
    unsigned long long v_clean;      // its rows past the end are zeros
    uint32_t tmem_base;
};

// ---- tcgen05 ---------------------------------------------------------------

// Shared-memory operand descriptor of the 128-byte swizzled layout: rows of
// 128 bytes, 8-row groups 1024 bytes apart (the stride field), 16-byte chunk
// c of row t stored at chunk c ^ (t mod 8).  The start address advances by
// 32 bytes per 16-element K step inside a 64-element half; every block
// starts on a 1024-byte boundary, so the base-offset field stays 0.  `lead`
// (the leading field) is the distance of neighbouring 64-element halves of an
// MN-major operand wider than 64.  Addresses are below 2^18, so a descriptor
// of the same layout `bytes` further is the sum with bytes / 16.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lead = 16) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// True on one lane of the (converged) warp.  What that thread does alone,
// descriptors included, then runs on the warp's uniform registers: with
// `lane == 0` instead, an MMA took 80 to 100 cycles to issue.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Instruction descriptor of kind::f16: fp32 accumulator, fp16 A and B, A
// K-major, B K-major or (mn_major) MN-major, M x N.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | (b_mn_major ? (1u << 16) : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}

// The same with A in tensor memory: row m of A in lane m, 16-bit elements
// two per column from a_tmem on.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
        : "memory");
}

// The mbarrier gets one arrival when every MMA this thread issued so far has
// completed.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define PKV_R8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                  "=r"(v[i + 6]), "=r"(v[i + 7])
#define PKV_W8(i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), \
                  "r"(v[i + 6]), "r"(v[i + 7])

// Lane l of the warp reads lane (32 (warp mod 4) + l) of tensor memory,
// columns col .. col + 31 (resp. 15); complete with tmem_ld_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : PKV_R8(0), PKV_R8(8), PKV_R8(16), PKV_R8(24)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : PKV_R8(0), PKV_R8(8)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        PKV_W8(0), PKV_W8(8), PKV_W8(16), PKV_W8(24)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        PKV_W8(0), PKV_W8(8)
        : "memory");
}
#undef PKV_R8
#undef PKV_W8
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bounded wait on an mbarrier phase by every lane of the warp (each lane
// observes the completion itself; cheaper than one lane polling and a
// broadcast when the phase has already completed); true on every lane only
// if it completed for all of them, so the warp leaves its loops together.
__device__ __forceinline__ bool wait_lanes(uint32_t bar, uint32_t parity, int *status) {
    return __all_sync(FULL, mbar_wait(bar, parity, status));
}

// Packed pairs of fp32 for Blackwell's two-wide add.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 4-D tiled TMA load (no cache hint): K/V tiles are read again by the other
// query tiles of the same head, so they keep the default L2 policy.
__device__ __forceinline__ void tma_load_4d_plain(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                  int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// Byte offset of 16-byte chunk c (elements 8c .. 8c + 7) of row t in a block
// of `rows` rows stored as 64-element halves, each half [rows][128 bytes]
// swizzled.
__device__ __forceinline__ uint32_t swz(int t, int c, int rows) {
    return (uint32_t)((((c >> 3) * rows + t) << 7) + (((c & 7) ^ (t & 7)) << 4));
}

// 16-byte cp.async that reads `bytes` (16 or 0) and zero-fills the rest.
__device__ __forceinline__ void cp_async16_zfill(uint32_t smem, const void *gmem, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t smem, const void *gmem, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}

template <int D, bool CAUSAL, bool Q8, bool SPLIT>
__global__ void __launch_bounds__(NTHREADS, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const Params p) {
    using C = Cfg<D, Q8>;
    constexpr int BN = C::BN;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);

    // Work item, the longest first.  Causal: the last query tiles.  Cross: the
    // longest contexts -- with blocks taken in the order of the sequences, four
    // prompts' 384 blocks on 152 SMs left 40 % of the time idle behind the long
    // ones (batches of up to kOrderSeqs with room for long contexts: each block
    // ranks the lengths itself, which takes it about a microsecond).
    const int part = SPLIT ? (int)blockIdx.x % p.splits : 0;
    const int b = SPLIT ? (int)blockIdx.x / p.splits : (int)blockIdx.x;
    int qp = p.n_qp - 1 - b / p.n_items;
    int item = b - (b / p.n_items) * p.n_items;
    if constexpr (!CAUSAL) {
        const int per = p.n_kv_heads * p.n_qp;
        int seq = b / per;
        if (p.n_seqs > 1 && p.n_seqs <= kOrderSeqs && p.max_blocks * p.block_size >= kOrderContext) {
            __shared__ int len_of[kOrderSeqs];
            __shared__ int picked;
            const int u = (int)threadIdx.x;
            const int mine = u < p.n_seqs ? p.lens[u] : 0;
            if (u < p.n_seqs) len_of[u] = mine;
            __syncthreads();
            if (u < p.n_seqs) {
                int rank = 0;
                for (int v = 0; v < p.n_seqs; ++v) rank += len_of[v] > mine || (len_of[v] == mine && v < u);
                if (rank == seq) picked = u;
            }
            __syncthreads();
            seq = picked;
        }
        qp = b % per / p.n_kv_heads;
        item = seq * p.n_kv_heads + b % p.n_kv_heads;
    }
    const int s = item / p.n_kv_heads;
    const int h = item - s * p.n_kv_heads;
    const int warp = (int)threadIdx.x / 32;
    const int lane = (int)threadIdx.x % 32;
    const int maxctx = p.max_blocks * p.block_size;

    // Loaders: the block ids of their first tiles (what of the table row that
    // needs, whatever it holds), on the way together with the lengths.
    const bool loader = warp >= LOAD_WARP0 && warp < LOAD_WARP0 + 4;
    const bool is_v = warp >= LOAD_WARP0 + 2;
    const int li = (warp - LOAD_WARP0) & 1;                  // this warp's boxes: lane % 2 == li
    const int32_t *bt_row = p.bt + (size_t)s * p.max_blocks;
    constexpr int CPR = D / 16;                              // e4m3: chunks of a row of codes
    constexpr int TPI = 32 / CPR;                            // tokens of a warp per chunk index
    constexpr int TW = BN / 2;                               // tokens of a warp
    constexpr int IDS = TW / 32;
    auto tile_token = [&](int lt) { return lt / TPI * (2 * TPI) + li * TPI + lt % TPI; };
    int first_id[2] = {0, 0};
    auto first_look = [&](int from) {
        const int page = p.block_size >= 16 ? p.block_shift : 0;
#pragma unroll
        for (int k = 0; k < (Q8 ? IDS : 2); ++k) {
            const int tok = from + (Q8 ? tile_token(lane + 32 * k) : k * BN + lane * p.box_rows);
            first_id[k] = bt_row[min(tok >> page, p.max_blocks - 1)];
        }
    };
    if (!SPLIT && loader) first_look(0);

    // lengths and new-token counts, clamped (and flagged) to what the table
    // and the call allow
    int L = p.lens[s];
    const bool flagger = threadIdx.x == 0 && qp == 0 && h == 0;
    if (L < 0 || L > maxctx) {
        if (flagger) atomicOr(p.status, PF_DEV_BAD_LENGTH);
        L = L < 0 ? 0 : maxctx;
    }
    const int q0 = CAUSAL || p.cu_q ? p.cu_q[s] : s;
    int n = CAUSAL || p.cu_q ? p.cu_q[s + 1] - q0 : 1;
    if (n < 0 || (CAUSAL && n > L) || n > p.max_new) {
        if (flagger) atomicOr(p.status, PF_DEV_BAD_LENGTH);
        n = n < 0 ? 0 : min(CAUSAL ? min(n, L) : n, p.max_new);
    }
    const int rows = n * p.gh;
    const int r0 = qp * 2 * QT;
    if (r0 >= rows) return;                  // the whole CTA: no row here
    const int r_end = min(r0 + 2 * QT, rows);
    if (SPLIT && L == 0 && part > 0) return;
    if (!CAUSAL && L == 0) {                 // nothing to attend to: zeros
        const size_t o0 = ((size_t)q0 * p.n_q_heads + (size_t)h * p.gh) * D;
        for (int e = threadIdx.x; e < (r_end - r0) * (D / 8); e += NTHREADS) {
            const int r = r0 + e / (D / 8);
            const size_t o = o0 + ((size_t)(r / p.gh) * p.n_q_heads + r % p.gh) * D + e % (D / 8) * 8;
            if (p.out_f32) {
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + o);
                dst[0] = dst[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<__half *>(p.out) + o) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }
    const int base = L - n;                  // position of new token 0 (causal)
    // per query tile: its last position and its number of K/V tiles
    int nt[2], pmax[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int gr0 = r0 + g * QT;
        if (gr0 >= r_end) {
            nt[g] = 0;
            pmax[g] = 0;
        } else {
            pmax[g] = CAUSAL ? base + (min(gr0 + QT, r_end) - 1) / p.gh : L - 1;
            nt[g] = pmax[g] / BN + 1;
        }
    }
    int p_max = max(pmax[0], pmax[1]);
    int ntt = max(nt[0], nt[1]);
    // This CTA's part of the context: tokens tok0 .. tok0 + p_max; positions
    // and tiles count from tok0.
    int tok0 = 0, n_parts = 1;
    if constexpr (SPLIT) {
        const int per = part_tiles(ntt, p.splits);
        n_parts = (ntt + per - 1) / per;
        if (part >= n_parts) return;
        tok0 = part * per * BN;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            pmax[g] = min(pmax[g], tok0 + per * BN - 1) - tok0;
            nt[g] = nt[g] == 0 || pmax[g] < 0 ? 0 : pmax[g] / BN + 1;
        }
        p_max = max(pmax[0], pmax[1]);
        ntt = max(nt[0], nt[1]);
        if (loader) first_look(tok0);
    }

    const uint32_t s_k = smem_addr(sm + C::OFF_K);
    const uint32_t s_v = smem_addr(sm + C::OFF_V);
    auto bar = [](unsigned long long &x) { return smem_addr(&x); };

    // Row r0 + d of the CTA: its new token, and where it lies in q and out.
    // d + r0 mod gh is below 272, where the product with 65536 / gh (rounded
    // up) gives the quotient.
    const int i0 = r0 / p.gh, rem0 = r0 - i0 * p.gh;
    auto token_of = [&](int d) { return i0 + (((rem0 + d) * p.gh_magic) >> 16); };
    auto row_at = [&](int d) {
        const int i = token_of(d);
        return ((size_t)(q0 + i) * p.n_q_heads + (size_t)h * p.gh + (rem0 + d - (i - i0) * p.gh)) * D;
    };
    // Softmax threads: the query rows into shared memory (zeros past the last
    // row), 16 bytes each and neighbouring lanes neighbouring chunks, before
    // the setup barrier, which then orders them before the first MMA.
    const int g = (warp / 4) & 1;
    const int t = (int)threadIdx.x % 128;                    // row of the tile = tensor-memory lane
    const bool valid = warp < SOFTMAX_WARPS && r0 + g * QT + t < r_end;
    const int lim = CAUSAL && valid ? base + token_of(g * QT + t) - tok0 : pmax[g];   // last position this row sees
    if (warp < SOFTMAX_WARPS) {
        constexpr int CH = D / 8;
#pragma unroll
        for (int it = 0; it < CH; ++it) {
            const int d = it * (256 / CH) + (int)threadIdx.x / CH, c = (int)threadIdx.x % CH;
            const bool ok = r0 + d < r_end;
            cp_async16_zfill(smem_addr(sm) + (d / QT) * C::Q_BYTES + swz(d % QT, c, QT),
                             p.q + (ok ? row_at(d) + c * 8 : 0), ok ? 16u : 0u);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_shared();
    }
    // Loaders: block id of box `lane` of tile j (pages of 16 tokens and
    // more; boxes past the CTA's last position are not loaded), read two
    // tiles ahead of its use and range-checked only when used.
    const int box = p.box_rows;
    auto n_boxes = [&](int j) { return min(BN / box, (p_max - j * BN) / box + 1); };
    auto raw_id = [&](int j) {
        return (!Q8 && p.block_size >= 16 && j < ntt && lane < n_boxes(j)) ? bt_row[(tok0 + j * BN + lane * box) / p.block_size] : 0;
    };
    // Loaders (two warps for K, two for V, each issuing every other page
    // box of a tile; a stage is refilled once the MMAs of the tile that used
    // it -- the scores for K, the products for V -- are done).  They set up
    // their barriers and stage tile 0 before the setup barrier, so the first
    // tiles arrive while the query rows load.
    const CUtensorMap *map = is_v ? &tmv : &tmk;
    unsigned long long *full = is_v ? bars.v_full : bars.k_full;
    unsigned long long *empty = is_v ? bars.v_empty : bars.k_empty;
    const uint32_t s_base = is_v ? s_v : s_k;
    const __half *pool_base = static_cast<const __half *>(is_v ? p.v_pool : p.k_pool);
    const int B = p.block_size;
    int issued = 0;
    // tile j into its stage (box `lane` from block id `id`); false if a wait ran out
    auto load_tile = [&](int j, int id) -> bool {
        const int st = j % NS;
        const uint32_t dst = s_base + st * C::KV_BYTES;
        if (j >= NS && !wait_lanes(bar(empty[st]), ((j / NS) - 1) & 1, p.status)) return false;
        if (B >= 16) {
            const int nb = n_boxes(j);
            const bool mine = lane < nb && (lane & 1) == li;
            if (mine && (id < 0 || id >= p.n_blocks)) {
                atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                id = 0;
            }
            if (lane == 0) mbar_arrive_expect_tx(bar(full[st]), (uint32_t)((nb + 1 - li) / 2) * box * D * 2);
            __syncwarp();
            if (mine) {
                const int row = (int)(p.layer_row0 + (long long)id * B + (tok0 + j * BN + lane * box) % B);
#pragma unroll
                for (int hf = 0; hf < C::HALVES; ++hf)
                    tma_load_4d_plain(dst + (uint32_t)(hf * BN + lane * box) * 128u, map, 0, row, hf, h, bar(full[st]));
            }
        } else {
            // one token per page: 16-byte cp.async per chunk into its
            // swizzled place, then a proxy fence before the arrival
            for (int tk = lane + 32 * li; tk < BN; tk += 64) {
                const int tok = j * BN + tk;
                if (tok > p_max) break;
                int bid = bt_row[tok0 + tok];
                if (bid < 0 || bid >= p.n_blocks) {
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
        ++issued;
        return true;
    };
    // e4m3: the tile's 512 16-byte chunks are dealt to the 64 lanes of the
    // tensor's two warps; chunk i of a lane is of token 2 TPI i + TPI li +
    // lane / CPR.  Lane l looks up the block ids (one tile ahead of their
    // copy) and copies the scales of the warp's tokens l, l + 32 (in order).
    const uint32_t raw = smem_addr(sm + C::OFF_RAW) + (is_v ? kRawStages * C::RAW_BYTES : 0);
    const float *scale_base = is_v ? p.v_scale : p.k_scale;
    int q_id[IDS];                                           // raw ids of the next tile to copy (-2: no token)
    auto q8_look_up = [&](int j) {
#pragma unroll
        for (int k = 0; k < IDS; ++k) {
            const int tok = j * BN + tile_token(lane + 32 * k);
            q_id[k] = tok <= p_max ? bt_row[(tok0 + tok) >> p.block_shift] : -2;
        }
    };
    // this lane's chunk 0 in a raw stage, in the pool and in a swizzled stage;
    // chunk i is 2 TPI tokens further (t mod 8, the swizzle, stays)
    const int x0 = li * TPI + lane / CPR, c0 = lane % CPR;
    const uint32_t raw_at = (uint32_t)(x0 * CPR + c0) * 16;
    const uint32_t row_bytes = (uint32_t)p.n_kv_heads * D;
    const uint8_t *codes = reinterpret_cast<const uint8_t *>(pool_base) + h * D + c0 * 16;
    const uint32_t wide_at[2] = {swz(x0, 2 * c0, BN), swz(x0, 2 * c0 + 1, BN)};
    auto q8_copy = [&](int j) {                              // tile j into raw stage j mod kRawStages
        const uint32_t dst = raw + (uint32_t)(j % kRawStages) * C::RAW_BYTES;
        if (j < ntt) {
            int row[IDS];
            bool whole = true;
#pragma unroll
            for (int k = 0; k < IDS; ++k) {
                const int id = q_id[k], lt = lane + 32 * k;
                const bool ok = (unsigned)id < (unsigned)p.n_blocks;
                if (!ok && id != -2) atomicOr(p.status, PF_DEV_BAD_BLOCK_ID);
                row[k] = ok ? (int)p.layer_row0 + (id << p.block_shift) + ((tok0 + j * BN + tile_token(lt)) & (B - 1)) : -1;
                whole = whole && ok;
                cp_async4_zfill(dst + BN * D + (li * TW + lt) * 4,
                                scale_base + (ok ? (size_t)(unsigned)((int)p.layer_page0 + id) * p.n_kv_heads + h : 0),
                                ok ? 4u : 0u);
            }
            if (__all_sync(FULL, whole)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r8 = __shfl_sync(FULL, row[i * TPI / 32], i * TPI % 32 + lane / CPR);
                    cp_async16_cg(dst + raw_at + i * 2 * TPI * CPR * 16, codes + (size_t)(unsigned)r8 * row_bytes);
                }
            } else {                                          // the end, or bad ids: zeros
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r8 = __shfl_sync(FULL, row[i * TPI / 32], i * TPI % 32 + lane / CPR);
                    cp_async16_zfill(dst + raw_at + i * 2 * TPI * CPR * 16,
                                     codes + (r8 < 0 ? 0 : (size_t)(unsigned)r8 * row_bytes), r8 < 0 ? 0u : 16u);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (j + 1 < ntt) q8_look_up(j + 1);
    };
    // tile j from its raw stage into its swizzled stage; false if a wait ran out
    auto q8_widen = [&](int j) -> bool {
        const uint32_t src = raw + (uint32_t)(j % kRawStages) * C::RAW_BYTES;
        const int st = j % NS;
        const uint32_t dst = s_base + st * C::KV_BYTES;
        if (j >= NS && !wait_lanes(bar(empty[st]), ((j / NS) - 1) & 1, p.status)) return false;
        constexpr int AT_ONCE = D == 64 ? 2 : 4;
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += AT_ONCE) {
            uint4 w[AT_ONCE];
            float f[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                             : "r"(src + raw_at + (i0 + i) * 2 * TPI * CPR * 16));
                asm volatile("ld.shared.f32 %0, [%1];"
                             : "=f"(f[i])
                             : "r"(src + BN * D + (li * TW + (i0 + i) * TPI + lane / CPR) * 4));
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const __half2 f2 = __float2half2_rn(f[i]);
                const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
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
        return true;
    };
    int id0 = 0, id1 = 0;
    if (loader) {
        if (warp == LOAD_WARP0 && lane == 0) {
            // two loader warps arrive on each full barrier
            for (int k = 0; k < NS; ++k) {
                mbar_init(bar(bars.k_full[k]), !Q8 && B >= 16 ? 2u : 64u);
                mbar_init(bar(bars.v_full[k]), !Q8 && B >= 16 ? 2u : 64u);
                mbar_init(bar(bars.k_empty[k]), 1);
                mbar_init(bar(bars.v_empty[k]), 1);
            }
            mbar_init_fence();
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");   // the loader warps: barriers initialised
        // They need nothing that the other warps set up, which wait for these
        // barriers: they pass the setup barrier without waiting.
        __syncwarp();
        asm volatile("bar.arrive 2, %0;" ::"n"(NTHREADS) : "memory");
        if constexpr (Q8) {
#pragma unroll
            for (int k = 0; k < IDS; ++k) q_id[k] = tile_token(lane + 32 * k) <= p_max ? first_id[k] : -2;
        } else {
            prefetch_tensormap(map);
            id0 = first_id[0];
            id1 = first_id[1];
            if (B >= 16) {
                const int id = id0;
                id0 = id1;
                id1 = raw_id(2);
                load_tile(0, id);
            }
        }
    }

    if (warp == MMA_S_WARP) {
        if (lane == 0) {
            for (int u = 0; u < 2; ++u) {
                mbar_init(bar(bars.s_full[u]), 1);
                mbar_init(bar(bars.s_free[u]), 128);
                mbar_init(bar(bars.p_full[u]), 128);
                mbar_init(bar(bars.o_done[u]), 1);
            }
            mbar_init(bar(bars.mma_done[0]), 1);
            mbar_init(bar(bars.mma_done[1]), 1);
            mbar_init(bar(bars.v_last), 1);
            mbar_init(bar(bars.v_clean), 1);
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
    if (!loader) asm volatile("bar.sync 2, %0;" ::"n"(NTHREADS) : "memory");
    tc_after_sync();
    const uint32_t tmem = loader ? 0u : bars.tmem_base;
    if (warp >= SOFTMAX_WARPS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<D>::OTHER));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<D>::SOFTMAX));

    if (warp < SOFTMAX_WARPS) {
        // ---------------------------------------------------------- softmax
        const uint32_t lane_off = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + (uint32_t)(g * BN);
        const uint32_t t_o = tmem + lane_off + (uint32_t)(C::COL_O + g * D);
        const uint32_t t_p = tmem + lane_off + (uint32_t)(C::COL_P + g * (BN / 2));
        const float sl = p.scale_log2;
        float m = -INFINITY;                                   // reference maximum, log2 units
        float l = 0.0f;                                        // sum of the weights
        bool ok = true;
        for (int j = 0; j < nt[g]; ++j) {
            if (!wait_lanes(bar(bars.s_full[g]), j & 1, p.status)) {
                ok = false;
                break;
            }
            tc_after_sync();
            uint32_t x[BN];                                    // raw scores (fp32 bits)
#pragma unroll
            for (int q = 0; q < BN / 32; ++q) tmem_ld32(t_s + q * 32, x + q * 32);
            tmem_ld_wait();
            tc_before_sync();
            mbar_arrive(bar(bars.s_free[g]));                 // the MMA warp may overwrite S

            // causal limit: columns past it never count
            const int cl = lim - j * BN;
            if (cl < BN - 1) {
#pragma unroll
                for (int c = 0; c < BN; ++c)
                    if (c > cl) x[c] = 0xff800000u;             // -inf
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
                f = ex2(m - mt);                                // m = -inf gives 0
                m = mt;
                l *= f;
            }
            // weights 2^(s sl - m); their sum two at a time
            const float nm = -m;
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

            // the previous product has finished reading P and adding to O
            if (j > 0) {
                if (!wait_lanes(bar(bars.o_done[g]), (j - 1) & 1, p.status)) {
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
        if (ok && nt[g] > 0 && wait_lanes(bar(bars.o_done[g]), (nt[g] - 1) & 1, p.status)) {
            tc_after_sync();
            const bool whole = !SPLIT || n_parts == 1;       // else a part: unscaled, fp32
            const float inv = whole ? 1.0f / l : 1.0f;
            const size_t part_row = SPLIT ? (((size_t)item * p.n_qp + qp) * p.splits + part) * (2 * QT) : 0;
            if (!whole) p.part_ml[part_row + g * QT + t] = make_float2(m, l);
            // The warp's 32 rows, 128 bytes of each at a time, through its own
            // rows of the query tile (whose MMAs are done): stored by rows
            // straight from tensor memory, 16 bytes per lane and row, the
            // output took 5,000 cycles.
            const uint32_t stage = smem_addr(sm) + g * C::Q_BYTES;
            const int t0 = (warp % 4) * 32;
            auto store = [&](auto f32_c) {
                constexpr bool F32 = decltype(f32_c)::value;
                constexpr int DP = F32 ? 32 : 64;            // dims of 128 bytes
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += DP) {
#pragma unroll
                    for (int part = 0; part < DP / 32; ++part) {
                        uint32_t o[32];
                        tmem_ld32(t_o + c0 + part * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < (F32 ? 8 : 4); ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if constexpr (F32) w[k] = __float_as_uint(__uint_as_float(o[4 * e + k]) * inv);
                                else w[k] = pack_half2(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                                       __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                            }
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             stage + swz(t0 + lane, part * 4 + e, QT)),
                                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                         : "memory");
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int it = 0; it < 8; ++it) {
                        const int row = t0 + it * 4 + lane / 8, c = lane % 8, d = g * QT + row;
                        uint4 w;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                     : "r"(stage + swz(row, c, QT)));
                        if (SPLIT && !whole) {
                            if (F32 && r0 + d < r_end)
                                *reinterpret_cast<uint4 *>(p.part_o + (part_row + d) * D + c0 + c * 4) = w;
                        } else if (r0 + d < r_end) {
                            const size_t at = row_at(d) + c0;
                            if constexpr (F32) *reinterpret_cast<uint4 *>(static_cast<float *>(p.out) + at + c * 4) = w;
                            else *reinterpret_cast<uint4 *>(static_cast<__half *>(p.out) + at + c * 8) = w;
                        }
                    }
                    __syncwarp();
                }
            };
            if (p.out_f32 || !whole) store(std::true_type());
            else store(std::false_type());
        }
    } else if (loader) {
        // ---------------------------------------------------------- loaders
        if constexpr (Q8) {
#pragma unroll 1
            for (int j = 0; j < kRawStages - 1; ++j) q8_copy(j);
            for (int j = 0; j < ntt; ++j) {
                __syncwarp();                                  // the raw stage of tile j - 1 has been read
                q8_copy(j + kRawStages - 1);
                asm volatile("cp.async.wait_group %0;" ::"n"(kRawStages - 1) : "memory");
                __syncwarp();
                if (!q8_widen(j)) break;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        for (int j = Q8 ? ntt : issued; j < ntt; ++j) {
            int id = id0;
            id0 = id1;
            id1 = raw_id(j + 2);
            if (!load_tile(j, id)) break;
        }
        // copies still in flight (only after a wait ran out) land before the CTA exits
        if (!Q8 && B >= 16) {
            for (int j = max(0, issued - NS); j < issued; ++j) wait_lanes(bar(full[j % NS]), (j / NS) & 1, p.status);
        }
    } else if (warp == MMA_S_WARP) {
        // ------------------------------------------------- MMA: S = Q K^T
        constexpr uint32_t ID_S = idesc_f16(QT, BN, false);
        if (elect_one()) {
            const uint64_t dq = sdesc(smem_addr(sm)), dk = sdesc(s_k);
            bool ok = true;
            int st = 0, phase = 0;
            for (int j = 0; ok && j < ntt; ++j) {
                if (!mbar_wait(bar(bars.k_full[st]), phase, p.status)) break;
                for (int g = 0; g < 2; ++g) {
                    if (j >= nt[g]) continue;
                    // S of this query tile has been read (its previous tile)
                    if (j > 0 && !mbar_wait(bar(bars.s_free[g]), (j - 1) & 1, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_after_sync();
                    const uint64_t a = dq + g * (C::Q_BYTES / 16), b = dk + st * (C::KV_BYTES / 16);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma(tmem + g * BN, a + (kk / 4) * (QT * 128 / 16) + (kk % 4) * 2,
                             b + (kk / 4) * (BN * 128 / 16) + (kk % 4) * 2, ID_S, kk > 0);
                    umma_commit(bar(bars.s_full[g]));
                }
                if (ok) umma_commit(bar(bars.k_empty[st]));
                if (++st == NS) {
                    st = 0;
                    phase ^= 1;
                }
            }
            // every MMA issued has completed before tensor memory is released
            umma_commit(bar(bars.mma_done[0]));
        }
        __syncwarp();
        wait_lanes(bar(bars.mma_done[0]), 0, p.status);
    } else if (warp == MMA_PV_WARP) {
        // ------------------------------------------------ MMA: O += P V
        constexpr uint32_t ID_PV = idesc_f16(QT, D, true);
        if (elect_one()) {
            const uint64_t dv = sdesc(s_v, BN * 128);
            bool ok = true;
            int st = 0, phase = 0;
            for (int j = 0; ok && j < ntt; ++j) {
                if (!mbar_wait(bar(bars.v_full[st]), phase, p.status)) break;
                if (!Q8 && j == ntt - 1) {
                    mbar_arrive(bar(bars.v_last));
                    if (!mbar_wait(bar(bars.v_clean), 0, p.status)) break;
                }
                for (int g = 0; g < 2; ++g) {
                    if (j >= nt[g]) continue;
                    if (!mbar_wait(bar(bars.p_full[g]), j & 1, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_after_sync();
                    const uint64_t b = dv + st * (C::KV_BYTES / 16);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        umma_ts(tmem + C::COL_O + g * D, tmem + C::COL_P + g * (BN / 2) + kk * 8, b + kk * (2048 / 16),
                                ID_PV, j > 0 || kk > 0);
                    umma_commit(bar(bars.o_done[g]));
                }
                if (ok) umma_commit(bar(bars.v_empty[st]));
                if (++st == NS) {
                    st = 0;
                    phase ^= 1;
                }
            }
            umma_commit(bar(bars.mma_done[1]));
        }
        __syncwarp();
        wait_lanes(bar(bars.mma_done[1]), 0, p.status);
    } else if (!Q8 && warp == CLEAN_WARP) {
        // V rows past the CTA's last position: zeros (a zero weight times a
        // non-finite value would not vanish)
        if (wait_lanes(bar(bars.v_last), 0, p.status)) {
            uint8_t *vt = sm + C::OFF_V + (ntt - 1) % NS * C::KV_BYTES;
            const int first = p_max - (ntt - 1) * BN + 1;
            for (int e = lane; e < (BN - first) * 8 * C::HALVES; e += 32) {
                const int row = first + e / (8 * C::HALVES);
                const int rest = e % (8 * C::HALVES);
                *reinterpret_cast<uint4 *>(vt + ((rest / 8) * BN + row) * 128 + (rest % 8) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bars.v_clean));
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
// maximum m_i, out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over the parts
// that the row sees.  A warp per row; lane i holds part i's m and l.
constexpr int kMergeWarps = 8;
template <int D, bool CAUSAL>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_parts_kernel(const Params p) {
    constexpr int BN = Cfg<D, false>::BN;
    constexpr int V = D / 32;                // values of a lane
    const int blk = (int)blockIdx.x;
    const int item = blk / p.n_qp, qp = blk - item * p.n_qp;
    const int s = item / p.n_kv_heads, h = item - s * p.n_kv_heads;
    const int lane = (int)threadIdx.x % 32;
    const int d = (int)blockIdx.y * kMergeWarps + (int)threadIdx.x / 32;   // row of the block
    griddep_wait();
    const int L = min(max(p.lens[s], 0), p.max_blocks * p.block_size);
    const int q0 = CAUSAL || p.cu_q ? p.cu_q[s] : s;
    int n = CAUSAL || p.cu_q ? max(p.cu_q[s + 1] - q0, 0) : 1;
    n = min(CAUSAL ? min(n, L) : n, p.max_new);
    const int rows = n * p.gh, r0 = qp * 2 * QT, r = r0 + d;
    if (r >= rows || L == 0) return;
    // the block's tiles and parts, as the main kernel counts them
    const int base = L - n;
    const int last = CAUSAL ? base + (min(r0 + 2 * QT, rows) - 1) / p.gh : L - 1;
    const int ntt = last / BN + 1, per = part_tiles(ntt, p.splits);
    if (ntt <= per) return;                  // one part: written by the main kernel
    const int parts = (CAUSAL ? base + r / p.gh : L - 1) / (per * BN) + 1;   // that the row sees
    const size_t row = ((size_t)blk * p.splits) * (2 * QT) + d;
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < parts) ml = p.part_ml[row + (size_t)lane * (2 * QT)];
    float top = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
    const float w = ex2(ml.x - top);
    float l = w * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    const float *at = p.part_o + row * D + lane * V;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
        const float wi = __shfl_sync(FULL, w, i);
        float x[V];
        if constexpr (V == 2) {
            const float2 v = *reinterpret_cast<const float2 *>(at + (size_t)i * (2 * QT) * D);
            x[0] = v.x, x[1] = v.y;
        } else {
            const float4 v = *reinterpret_cast<const float4 *>(at + (size_t)i * (2 * QT) * D);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(wi, x[k], acc[k]);
    }
    const float inv = 1.0f / l;
    const int i = r / p.gh;
    const size_t out = ((size_t)(q0 + i) * p.n_q_heads + (size_t)h * p.gh + (r - i * p.gh)) * D + lane * V;
#pragma unroll
    for (int k = 0; k < V; k += 2) {
        if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + out + k) = make_float2(acc[k] * inv, acc[k + 1] * inv);
        else *reinterpret_cast<__half2 *>(static_cast<__half *>(p.out) + out + k) = __floats2half2_rn(acc[k] * inv, acc[k + 1] * inv);
    }
}

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

}  // namespace
}  // namespace prefill_tc

namespace prefill_tc {
namespace {

using KernelFn = void (*)(CUtensorMap, CUtensorMap, Params);

template <int D, bool SPLIT>
KernelFn pick(bool causal, bool q8) {
    if (q8) return causal ? prefill_tc_kernel<D, true, true, SPLIT> : prefill_tc_kernel<D, false, true, SPLIT>;
    if constexpr (SPLIT) return prefill_tc_kernel<D, false, false, true>;   // (causal fp16 contexts are not cut)
    else return causal ? prefill_tc_kernel<D, true, false, false> : prefill_tc_kernel<D, false, false, false>;
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
                  size_t ws_bytes) {
    const long long blocks = prefill_tc::blocks_of(pool, n_seqs, n_q_heads, max_new);
    if ((causal && pool->dtype == PF_F16) || blocks <= 0) return 1;
    const int BN = pool->head_dim == 64 ? prefill_tc::Cfg<64, false>::BN : prefill_tc::Cfg<128, false>::BN;
    const long long tiles = ((long long)max_blocks * pool->block_size + BN - 1) / BN;
    const long long room = ws_bytes < kWorkspaceFront ? 0 : (long long)((ws_bytes - kWorkspaceFront) / prefill_tc::part_bytes(pool->head_dim));   // parts that fit
    const long long n = std::min(std::min(std::min((long long)sms, room) / blocks, tiles / prefill_tc::kMinTiles),
                                 (long long)prefill_tc::kMaxParts);
    if (n < 2) return 1;
    const long long rows = std::min((long long)max_new * (n_q_heads / pool->n_kv_heads), 2ll * prefill_tc::QT);
    const double bytes = 2.0 * (double)(blocks * n * rows) * pool->head_dim * sizeof(float);
    return 0.9 * (double)(tiles - (tiles + n - 1) / n) > 4.0 + bytes / 5e6 ? (int)n : 1;
}

size_t prompt_workspace_bytes(const pf_pool *pool, bool causal, int n_seqs, int n_q_heads, int max_blocks, int max_new) {
    int sms = 0;
    if (n_seqs <= 0 || max_new <= 0 || n_q_heads <= 0 || n_q_heads % pool->n_kv_heads || max_blocks <= 0 ||
        device_sms(false, &sms) != PF_OK)
        return 0;
    // a part per SM, whatever the batch: a smaller one takes no more
    return prompt_splits(pool, causal, n_seqs, n_q_heads, max_blocks, max_new, sms, SIZE_MAX) == 1
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
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.splits = 1;
    p.part_ml = nullptr;
    p.part_o = nullptr;
    const long long blocks = n_items * n_qp;
    if (a.workspace) {
        int sms = 0;
        const int rc = device_sms(true, &sms);
        if (rc) return rc;
        p.splits = prompt_splits(pool, a.causal, a.n_seqs, a.n_q_heads, a.max_blocks, a.max_new, sms, a.ws_bytes);
        p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.workspace) + kWorkspaceFront);
        p.part_o = reinterpret_cast<float *>(p.part_ml + (size_t)blocks * p.splits * 2 * prefill_tc::QT);
    }
    const bool split = p.splits > 1;
    const prefill_tc::KernelFn fn =
        D == 64 ? (split ? prefill_tc::pick<64, true>(a.causal, q8) : prefill_tc::pick<64, false>(a.causal, q8))
                : (split ? prefill_tc::pick<128, true>(a.causal, q8) : prefill_tc::pick<128, false>(a.causal, q8));
    const int smem = D == 64 ? (q8 ? prefill_tc::Cfg<64, true>::SMEM : prefill_tc::Cfg<64, false>::SMEM)
                             : (q8 ? prefill_tc::Cfg<128, true>::SMEM : prefill_tc::Cfg<128, false>::SMEM);
    // once per device and kernel (setting it twice does no harm)
    static std::atomic<bool> ready[kMaxDevices][16];
    std::atomic<bool> &done = ready[dev][(D == 64) + 2 * a.causal + 4 * q8 + 8 * split];
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
        e = D == 64 ? (a.causal ? cudaLaunchKernelEx(&cfg, prefill_tc::merge_parts_kernel<64, true>, p)
                                : cudaLaunchKernelEx(&cfg, prefill_tc::merge_parts_kernel<64, false>, p))
                    : (a.causal ? cudaLaunchKernelEx(&cfg, prefill_tc::merge_parts_kernel<128, true>, p)
                                : cudaLaunchKernelEx(&cfg, prefill_tc::merge_parts_kernel<128, false>, p));
        if (e != cudaSuccess) return cuda_error(e, "pf_paged_prefill_attention: merge launch");
    }
    return PF_OK;
}

}  // namespace pkv
