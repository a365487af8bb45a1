// Attention of a sequence's last tokens over its 4-bit KV cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q k_j - max),  k_j = z + s c (per 64 entries), v_j likewise.
//
// The queries that share a kv head (heads / kv_heads of them for each of the T tokens) are the rows, in tiles
// of 8 NT. A warp takes blocks of 16 cached tokens and runs both products on mma.sync m16n8k16 with the rows as
// the instruction's 8 columns:
//   S^T [16 tokens, 8 rows] = C_K [16 tokens, D] Q^T, one accumulator per 64 entries, then s (.) + z sum(q) in fp32;
//   O^T [D, 8 rows] += V^T [D, 16 tokens] P^T [16 tokens, 8 rows].
// The cache's layout is that of the A operands, so codes go from memory to the instruction with no shuffle: a
// word is four pairs (entries of a token for K, two tokens of an entry for V). P^T is S^T's
// fragment transposed within the warp (movmatrix). With few rows its floor is HBM's.
// P and V enter their product rounded to fp16, half a step each, which is of the size of the result's own rounding (3.0e-4 to
// 3.5e-4 of it in the norm, 2.1e-4 of that the last rounding). P in two parts leaves 2.9e-4 and was too dear: 64 sequences of
// up to 8192 tokens 87.6 us against 79.2, 4 tokens over 131072 59.4 against 52.3. Scores, maxima, sums and O stay in fp32.
//
// Work is split evenly whatever the lengths: the visible blocks of all (sequence, kv head, row tile), in pairs, in a
// row are cut into equal ranges, one per CTA of a grid that fills the SMs once; every CTA finds its range from
// the lens itself. A CTA's four warps take the pairs of a range in turn, each through its own ring of bulk
// copies (a block is contiguous, 18 D bytes) and with its own running maximum, sum and O^T, and join them in
// shared memory. A (sequence, head, tile) that lies in one range is finished there; the pieces of one that
// crosses ranges go to the workspace and a second, small kernel joins them, in the order of the ranges. Where no (sequence,
// head, tile) can be long, by the table's width and the window, each has a CTA of its own instead.
// Measured (D = 128, one token, 4 heads per kv head): 64 sequences of up to 8192 tokens, 330 MB, 79 us (4.2 TB/s). Nothing is
// full: 57 % of the issue slots (300 warp instructions per block), 52 % of DRAM, 26 % of the tensor pipe; the rest is waiting, in
// the chains within a pair and in each segment's start and join, with 12 warps per SM.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "tern_cache.cuh"

namespace tern {
namespace {

using namespace kv;

constexpr int kSplitWarps = 4;             // warps of a CTA where segments are split
constexpr int kFewWarps = 8, kManyWarps = 16;   // and where each has a CTA of its own: many where every CTA has an SM to itself
                                           // (16 sequences of 8 kv heads, 300 tokens 7.3 us against 8.4, 1000 tokens 10.3 against
                                           // 13.4), few where not (64 sequences: 15.8 against 25.5, 26.2 against 35.6)
constexpr int kDirectUnits = 36;           // units of a segment up to which it has, whatever the segments' number: at 1000 tokens (32
                                           // units) it costs one sequence 3 % and saves more of them 3 to 24 %, at 2000 (63) it mostly
                                           // costs, between them is not measured (1 / 4 / 16 / 64 sequences of 8 kv heads:
                                           // 300 tokens 6.5 6.7 6.9 14.2 us against 8.3 8.8 10.4 16.5 split; 1000 tokens
                                           // 9.0 9.1 9.6 24.7 against 8.7 9.5 12.7 25.5; 2000 12.8 12.8 14.0 36.3
                                           // against 9.0 10.8 14.9 33.8)
constexpr int kPair = 2 * kTok;            // tokens of a unit of work: two blocks
constexpr int kSlots = 3;                  // units in a warp's ring
// What a (sequence, head, tile) costs beyond its units, in units: its queries, pages, first copies and join. Measured, 8 rows: 64
// sequences of up to 8192 tokens 85.2 us with 8, 80.3 with 12, 78.7 with 16; 16 rows: 4 tokens of 32 sequences of up to 4000
// 59.9 with 12, 57.4 with 16, 50.1 with 24, 51.6 with 32.
constexpr int setup_of(int nt) { return nt == 1 ? 16 : 24; }
constexpr int kMinUnits = 8;               // cost per CTA at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxScale = 1e4f;          // keeps scale q k of finite inputs finite
constexpr float kLift = 7.f, kSlack = 8.f; // a probability counts 2^kLift at the running maximum, and up to 2^kSlack more (raise)
constexpr float kNothing = -3.4e38f;       // the maximum of no scores: below any score, and finite, so that no difference is NaN

struct Desc {               // a (sequence, kv head, row tile) in pieces: where the first lies
    int b, h, rt, pieces;   // pieces < 2: nothing to join
    int cta, rows;          // rows of (b, h) that are written
};

struct Args {
    Pool pool;
    const __half* q;
    __half* o;
    const int32_t* lens;
    const int32_t* counts;
    int window, sinks;
    int setup;                  // cost of a segment beyond its units
    int B, T, heads, G, RT;     // G = heads per kv head, RT = row tiles
    float scale;                // of the exponents (to base 2), > 0
    float slack;                // kSlack / scale
    uint32_t sign;              // turns the queries' signs where the caller's scale is negative
    Desc* desc;                 // [ndesc]: by (sequence, head, tile) where these are fewer than the CTAs, else by CTA
    int ndesc;
    bool by_segment;
    float* part;                // [gridDim.x][2 (continued from the range before, or not)][rows][D + 4]: O, maximum, sum
    unsigned int* status;
};

template <int D, int NT>
constexpr int part_floats() { return 8 * NT * (D + 4); }

__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return as_u32(__floats2half2_rn(lo, hi)); }

// The four words (D = 128) or two (D = 64) of a lane.
template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    }
}

// A sequence's part of the work: its queries' places and the pairs of blocks that they see, as one list (the
// pairs of the always visible first tokens, then those of the window).
struct Seq {
    int cnt, first, last;       // queries; the tokens of the first and the last
    int blocks;                 // blocks 0 .. blocks - 1 may be read
    int sb, wb, n;              // pairs 0 .. sb - 1, then wb ..; n in all
    int setup;
    __device__ __forceinline__ int pair(int v) const { return v < sb ? v : wb + v - sb; }
    __device__ __forceinline__ int cost() const { return max(n, 1) + setup; }   // one unit at least, so that its rows are written
};

__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
    Seq s;
    s.setup = a.setup;
    const int len = max(0, __ldg(a.lens + b));
    s.cnt = a.counts ? min(max(__ldg(a.counts + b), 0), a.T) : a.T;
    s.first = len - s.cnt;
    s.last = len - 1;
    s.blocks = s.last < 0 ? 0 : int(min(int64_t(s.last / kTok + 1), a.pool.width * a.pool.per_page));
    s.sb = s.wb = s.n = 0;
    if (s.cnt == 0 || s.blocks == 0) return s;
    const int end = (s.blocks + 1) / 2;
    if (a.window > 0) {
        s.wb = int(min(max(int64_t(0), int64_t(s.first) - a.window + 1) / kPair, int64_t(end)));   // (a query may lie before token 0)
        s.sb = min(int((unsigned(a.sinks) + kPair - 1) / kPair), s.wb);
    }
    s.n = s.sb + end - s.wb;
    return s;
}

__device__ __forceinline__ bool sees(int pos, int j, int window, int sinks) {
    return j <= pos && (window <= 0 || j > pos - window || j < sinks);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D, int NT>
struct State {
    float m[NT][2], l[NT][2];   // of rows 2 q and 2 q + 1 of each 8: maximum of q k, sum of this lane's tokens alone
    float o[NT][D / 16][4];
};

// Scores q k of a block of 16 tokens in shared memory: s [8 rows][token g: rows 2q, 2q + 1; token g + 8: the same].
template <int D, int NT>
__device__ __forceinline__ void scores(const uint8_t* u, const uint32_t (&qf)[NT][D / 32][4], const float (&qx)[NT][2], float (&s)[NT][4]) {
    constexpr int W = D / 32, NG = D / kGrp;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    {
        uint32_t ka[W], kb[W];
        load_words(u + lane * W * 4, ka);
        load_words(u + (32 + lane) * W * 4, kb);
        // What is not s c q of the scores, z sum(q) - 64 s sum(q): a product in tf32, where s and z are exact. Its column q is
        // half q of the token's scales (s, z per 64 entries), against sum(q)'s upper part, column q + 4 against its lower.
        float a0 = 0.f, a1 = 0.f;
        const __half* ks = reinterpret_cast<const __half*>(u + k_scales(D));
        if (NG == 2 || q < 2) {
            a0 = __half2float(ks[g * 2 * NG + q]);
            a1 = __half2float(ks[(g + 8) * 2 * NG + q]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_1688_first(s[t], a0, a1, a0, a1, qx[t][0], qx[t][1]);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            float acc[NT][4];
#pragma unroll
            for (int j = 2 * n; j < 2 * n + 2; ++j) {
                const uint32_t a8 = ka[j] >> 8, b8 = kb[j] >> 8;
                const uint32_t A0[4] = {code_pair_64<0>(ka[j], a8), code_pair_64<0>(kb[j], b8), code_pair_64<1>(ka[j], a8),
                                        code_pair_64<1>(kb[j], b8)};
                const uint32_t A1[4] = {code_pair_64<2>(ka[j], a8), code_pair_64<2>(kb[j], b8), code_pair_64<3>(ka[j], a8),
                                        code_pair_64<3>(kb[j], b8)};
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (j == 2 * n) mma_first(acc[t], A0, qf[t][j][0], qf[t][j][1]);
                    else mma_next(acc[t], A0, qf[t][j][0], qf[t][j][1]);
                    mma_next(acc[t], A1, qf[t][j][2], qf[t][j][3]);
                }
            }
            const float s0 = __half2float(ks[(g * NG + n) * 2]), s1 = __half2float(ks[((g + 8) * NG + n) * 2]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] += (i < 2 ? s0 : s1) * acc[t][i];
        }
    }
}

// Masks a block of which some row does not see some token, j0 the first token (or none is there): the scores, and in shared
// memory the scales of V's tokens that no row sees or that are not finite, which then count as zeros in the product; a row that
// sees one of the latter becomes NaN through its sum instead.
template <int D, int NT>
__device__ __forceinline__ void hide(uint8_t* u, int j0, bool there, const int (&pos)[NT][2], const Args& a, float (&s)[NT][4]) {
    constexpr int NG = D / kGrp;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    __half* vh = reinterpret_cast<__half*>(u + v_scales(D));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        bool odd = false, used = false;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) odd |= !(fabsf(__half2float(vh[((g >> 1) * NG + n) * 8 + z * 4 + 2 * h + (g & 1)])) < INFINITY);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (!there || !sees(pos[t][c], j0 + 8 * h + g, a.window, a.sinks)) s[t][2 * h + c] = -INFINITY;
                else {
                    used = true;
                    if (odd) s[t][2 * h + c] = NAN;
                }
            }
        const unsigned kept = __ballot_sync(0xffffffffu, used && !odd) >> (lane & ~3) & 0xFu;      // of the token's four lanes
        if (!kept && q < NG) {
            __half* at = vh + ((g >> 1) * NG + q) * 8 + 2 * h + (g & 1);
            at[0] = at[4] = __ushort_as_half(0);
        }
    }
}

// The running maximum of a row moves only when some token is 2^kSlack above it: seldom, so the reduction over the 8 lanes of
// a column is not paid per block. A probability counts 2^kLift at the maximum, so that P uses fp16's range up to 2^15: one of 2^-21
// of the maximum still has all its bits, and none above 2^-32 of it is lost. (Where a first token takes nearly all of the mass and
// has a small V, the result is left to such tokens.)
template <int D, int NT, int kBlocks>
__device__ __forceinline__ void raise(const float (&s)[kBlocks][NT][4], const Args& a, State<D, NT>& st) {
    bool up = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float top = fmaxf(s[0][t][c], s[0][t][2 + c]);
#pragma unroll
            for (int k = 1; k < kBlocks; ++k) top = fmaxf(top, fmaxf(s[k][t][c], s[k][t][2 + c]));
            up |= top - st.m[t][c] > a.slack;
        }
    if (!__any_sync(0xffffffffu, up)) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float m = st.m[t][c];
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) m = fmaxf(m, fmaxf(s[k][t][c], s[k][t][2 + c]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float f = m > st.m[t][c] ? ex2((st.m[t][c] - m) * a.scale) : 1.f;
            st.m[t][c] = m;
            st.l[t][c] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                st.o[t][i][c] *= f;
                st.o[t][i][2 + c] *= f;
            }
        }
}

// A block's probabilities, and its V into O^T. A score's distance to the maximum is taken before it is scaled: the product of
// a large score is off by more than the distance (scores past 2^28 gave infinities).
template <int D, int NT>
__device__ __forceinline__ void add_values(const uint8_t* u, const float (&s)[NT][4], const Args& a, State<D, NT>& st) {
    constexpr int W = D / 32, NG = D / kGrp;
    const int lane = threadIdx.x & 31, q = lane & 3;
    uint32_t b0[NT], b1[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ex2(fmaf(s[t][i] - st.m[t][i & 1], a.scale, kLift));
        st.l[t][0] += p[0] + p[2];
        st.l[t][1] += p[1] + p[3];
        b0[t] = transposed(pack_h2(p[0], p[1]));
        b1[t] = transposed(pack_h2(p[2], p[3]));
    }
    uint32_t va[W], vb[W];
    load_words(u + v_codes(D) + lane * W * 4, va);
    load_words(u + v_codes(D) + (32 + lane) * W * 4, vb);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        // steps and zeros of the lane's V tokens 2q, 2q + 1 and 2q + 8, 2q + 9
        const uint4 v = *reinterpret_cast<const uint4*>(u + v_scales(D) + (q * NG + n) * 16);
        const __half2 s0 = as_h2(v.x), s1 = as_h2(v.y), z0 = as_h2(v.z), z1 = as_h2(v.w);
#pragma unroll
        for (int j = 2 * n; j < 2 * n + 2; ++j) {
            const uint32_t a8 = va[j] >> 8, b8 = vb[j] >> 8;
            const uint32_t A0[4] = {as_u32(__hfma2(as_h2(code_pair<0, 0>(va[j], a8)), s0, z0)),
                                    as_u32(__hfma2(as_h2(code_pair<1, 0>(va[j], a8)), s0, z0)),
                                    as_u32(__hfma2(as_h2(code_pair<0, 0>(vb[j], b8)), s1, z1)),
                                    as_u32(__hfma2(as_h2(code_pair<1, 0>(vb[j], b8)), s1, z1))};
            const uint32_t A1[4] = {as_u32(__hfma2(as_h2(code_pair<2, 0>(va[j], a8)), s0, z0)),
                                    as_u32(__hfma2(as_h2(code_pair<3, 0>(va[j], a8)), s0, z0)),
                                    as_u32(__hfma2(as_h2(code_pair<2, 0>(vb[j], b8)), s1, z1)),
                                    as_u32(__hfma2(as_h2(code_pair<3, 0>(vb[j], b8)), s1, z1))};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mma_next(st.o[t][2 * j], A0, b0[t], b1[t]);
                mma_next(st.o[t][2 * j + 1], A1, b0[t], b1[t]);
            }
        }
    }
}

// The lane with `who` announces `expect` bytes on the barrier and starts a bulk copy of `bytes` (0: none).
__device__ __forceinline__ void bulk_pair(bool who, uint32_t expect, uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p, c;\n\t"
        "setp.ne.u32 p, %0, 0;\n\t"
        "setp.ne.and.u32 c, %4, 0, p;\n\t"
        "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], %1;\n\t"
        "@c cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%2], [%3], %4, [%5];\n\t}" ::"r"(uint32_t(who)),
        "r"(expect), "r"(to), "l"(reinterpret_cast<uint64_t>(from)), "r"(bytes), "r"(bar)
        : "memory");
}

// A second copy on a barrier that expects its bytes already.
__device__ __forceinline__ void bulk_more(bool who, uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %0, 0;\n\t"
        "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2], %3, [%4];\n\t}" ::"r"(uint32_t(who)),
        "r"(to), "l"(reinterpret_cast<uint64_t>(from)), "r"(bytes), "r"(bar)
        : "memory");
}

// Inclusive sum over the CTA's threads; total: over all of them. `sums` holds kWarps values and is free again
// after the next barrier.
template <int kWarps>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) v += sums[w];
        total += sums[w];
    }
    __syncthreads();
    return v;
}

template <int D, int NT, int kWarps>
struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = D + 4;                               // 16-byte rows; a fragment's stores hit all banks once
    static constexpr int ring_bytes = kSlots * 2 * unit_bytes(D);      // of a warp; its O^T after the last unit
    static_assert(kRows * kPitch * 4 <= ring_bytes, "a warp's rows fit its ring");
    alignas(128) uint8_t ring[kWarps][ring_bytes];
    uint64_t full[kWarps][kSlots];
    int64_t sums[kWarps];
    int64_t off;
    int b;
    float m[kWarps][kRows], l[kWarps][kRows], top[kRows];
};

// CTAs of an SM: what leaves each split variant its registers without spills. (D = 128, 8 rows: four CTAs of 128 registers took
// as long over long sequences and longer over short ones, 4 sequences of up to 4000 tokens 13.3 us against 12.0; 16 rows: three took
// 65.5 us over 131072 tokens against 61.1.) The direct ones of D = 128 and 8 rows have 128 registers and spill 24 bytes.
constexpr int resident(int D, int nt, int direct) { return direct ? (nt == 1 && direct == kFewWarps ? 2 : 1) : (nt == 1 ? 4 : 3) - (D == 128); }

// kDirect > 0: CTA i, of so many warps, takes the whole of segment i, and nothing is split or joined.
template <int D, int NT, int kDirect>
__global__ void __launch_bounds__((kDirect ? kDirect : kSplitWarps) * 32, resident(D, NT, kDirect))
    attention_kernel(const Args a) {
    constexpr int kWarps = kDirect ? kDirect : kSplitWarps, kThreads = kWarps * 32;
    using S = Smem<D, NT, kWarps>;
    constexpr int W = D / 32, NG = D / kGrp, kRows = 8 * NT, U = unit_bytes(D);   // U: bytes of a block
    extern __shared__ __align__(128) uint8_t raw[];
    S& sm = *reinterpret_cast<S*>(raw);
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kSlots; ++i) mbar_init(&sm.full[0][i], 1);
        fence_barrier_init();
    }
    __syncthreads();            // every warp uses its barriers from its first copy on
    grid_launch_dependents();
    grid_dependency_wait();

    // ---- this CTA's range of the cost of all (sequence, head, tile)
    const int per_seq = a.pool.heads * a.RT;
    int b, ht, c0;              // sequence; head and tile; how much of their cost lies before this range
    int64_t quota = 0, left;
    Seq seq;
    if (kDirect) {
        b = int(blockIdx.x) / per_seq;
        ht = int(blockIdx.x) % per_seq;
        seq = seq_of(a, b);
        c0 = 0;
        left = seq.cost();
    } else {
        int64_t total = 0, mine = 0, incl = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + threadIdx.x;
            mine = b < a.B ? int64_t(seq_of(a, b).cost()) * per_seq : 0;
            int64_t t;
            incl = total + block_scan<kWarps>(mine, sm.sums, t);
            total += t;
        }
        quota = max((total + gridDim.x - 1) / gridDim.x, int64_t(kMinUnits));
        const int64_t u0 = int64_t(blockIdx.x) * quota;
        if (u0 >= total) {
            if (threadIdx.x == 0 && !a.by_segment) a.desc[blockIdx.x].pieces = 0;
            return;
        }
        if (a.B <= kThreads) {
            if (mine && incl - mine <= u0 && u0 < incl) {
                sm.b = threadIdx.x;
                sm.off = u0 - (incl - mine);
            }
        } else {
            int64_t before = 0;
            for (int b0 = 0; b0 < a.B; b0 += kThreads) {
                const int b = b0 + threadIdx.x;
                mine = b < a.B ? int64_t(seq_of(a, b).cost()) * per_seq : 0;
                int64_t t;
                incl = before + block_scan<kWarps>(mine, sm.sums, t);
                if (mine && incl - mine <= u0 && u0 < incl) {
                    sm.b = b;
                    sm.off = u0 - (incl - mine);
                }
                before += t;
                if (before > u0) break;
            }
        }
        __syncthreads();
        b = sm.b;
        seq = seq_of(a, b);
        ht = int(sm.off / seq.cost());                         // head and tile
        c0 = int(sm.off - int64_t(ht) * seq.cost());       // and how much of its cost lies before this range
        left = min(quota, total - u0);
    }
    Desc cut{0, 0, 0, 0, 0, 0};    // the segment that goes on behind this range, if it begins in it
    const bool odd_page = a.pool.per_page & 1;             // a pair may lie in two pages
    uint64_t* full = sm.full[warp];
    uint8_t* ring = sm.ring[warp];
    const uint32_t ring_at = smem_u32(ring), full_at = smem_u32(full);
    uint32_t slot = 0, phase = 0;      // of the next unit this warp waits for, over all segments
    bool ok = true;

    while (left > 0) {
        const int h = ht / a.RT, r0 = (ht % a.RT) * kRows;
        const int c1 = int(min(int64_t(seq.cost()), c0 + left));
        const int v0 = max(0, c0 - a.setup), v1 = max(0, c1 - a.setup);   // units of this range
        if (v1 > 0) {
        const int rows = seq.cnt * a.G;                    // of this sequence and head; the tile's are r0 ..
        const bool live = r0 < rows && seq.n > 0;
        // ---- the warp's units v0 + warp, + kWarps, ..; lane i looks up the pages of the i-th of each 32: the block's place in
        // the pool, and two ballots for which of its blocks there are
        const int n = live ? (v1 - v0 - warp + kWarps - 1) / kWarps : 0;
        uint32_t at0 = 0, at1 = 0, have0 = 0, have1 = 0;
        uint32_t present = 0;          // two bits per slot
        auto look = [&](int i0) {
            const int blk = 2 * seq.pair(v0 + warp + (i0 + lane) * kWarps);
            const bool want = i0 + lane < n;
            const int p0 = want ? a.pool.place(b, h, blk) : -1;
            const int p1 = !want || blk + 1 >= seq.blocks ? -1 : !odd_page ? p0 : a.pool.place(b, h, blk + 1);
            at0 = uint32_t(p0), at1 = uint32_t(p1);
            have0 = __ballot_sync(0xffffffffu, p0 >= 0);
            have1 = __ballot_sync(0xffffffffu, p1 >= 0);
        };
        auto issue = [&](int i, uint32_t slot) {
            if ((i & 31) == 0) look(i);
            const unsigned h0 = have0 >> (i & 31) & 1u, h1 = have1 >> (i & 31) & 1u;
            present = (present & ~(3u << (2 * slot))) | (h0 | h1 << 1) << (2 * slot);
            const uint32_t p0 = __shfl_sync(0xffffffffu, at0, i & 31);
            const uint32_t to = ring_at + slot * 2 * U, bar = full_at + slot * 8;
            const uint32_t bytes = (h0 + h1) * U;
            if (!odd_page) {
                bulk_pair(lane == 0, bytes, to, a.pool.pool + uint64_t(p0) * U, bytes, bar);
            } else {
                const uint32_t p1 = __shfl_sync(0xffffffffu, at1, i & 31);
                bulk_pair(lane == 0, bytes, to, a.pool.pool + uint64_t(p0) * U, h0 * U, bar);
                bulk_more(lane == 0 && h1, to + U, a.pool.pool + uint64_t(p1) * U, U, bar);
            }
        };
        int issued = 0;
        for (uint32_t at = slot; issued < n && issued < kSlots && ok; ++issued) {
            issue(issued, at);
            at = at == kSlots - 1 ? 0 : at + 1;
        }

        // ---- the tile's queries: row R is token R / G, head R % G of the kv head
        auto row_at = [&](int R) { return ((int64_t(b) * a.T + R / a.G) * a.heads + h * a.G + R % a.G) * D; };
        uint32_t qf[NT][W][4];
        float qx[NT][2];
        int pos[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float part[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) part[i] = 0.f;
            const int R = r0 + 8 * t + g;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint4 v = R < rows && n > 0 ? *reinterpret_cast<const uint4*>(a.q + row_at(R) + 32 * j + 8 * q) : make_uint4(0, 0, 0, 0);
                qf[t][j][0] = v.x ^ a.sign, qf[t][j][1] = v.y ^ a.sign, qf[t][j][2] = v.z ^ a.sign, qf[t][j][3] = v.w ^ a.sign;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __half22float2(as_h2(qf[t][j][i]));
                    part[j / 2] += f.x + f.y;
                }
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                part[i] += __shfl_xor_sync(0xffffffffu, part[i], 1);
                part[i] += __shfl_xor_sync(0xffffffffu, part[i], 2);
            }
            // of row g: -64 sum(q) against the steps (even columns), sum(q) against the zeros
            const float mine = NG == 2 && q >= 2 ? part[NG - 1] : part[0];
            const float v = NG == 2 || q < 2 ? (q & 1 ? mine : -64.f * mine) : 0.f;
            qx[t][0] = tf32_part(v);
            qx[t][1] = tf32_part(v - qx[t][0]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int Rc = r0 + 8 * t + 2 * q + c;
                pos[t][c] = Rc < rows ? seq.first + Rc / a.G : -1;
            }
        }
        const int tile_first = seq.first + r0 / a.G, tile_last = seq.first + (min(r0 + kRows, rows) - 1) / a.G;
        State<D, NT> st;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            st.m[t][0] = st.m[t][1] = kNothing;
            st.l[t][0] = st.l[t][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) st.o[t][i][0] = st.o[t][i][1] = st.o[t][i][2] = st.o[t][i][3] = 0.f;
        }
        // units [whole0, whole1) and [0, sink1) of the list: every row sees every token
        const int whole1 = seq.sb + max(0, (tile_first + 1) / kPair - seq.wb);
        const int whole0 = a.window > 0 ? seq.sb + max(0, int(max(int64_t(0), int64_t(tile_last) - a.window + kPair) / kPair) - seq.wb) : 0;
        const int sink1 = a.window > 0 ? min(seq.sb, min(a.sinks, tile_first + 1) / kPair) : 0;
        for (int i = 0; i < n; ++i) {
            ok = ok && mbar_wait(&full[slot], phase);
            const int v = v0 + warp + i * kWarps;
            const unsigned have = present >> (2 * slot) & 3u;
            const bool whole = have == 3u && ((v >= whole0 && v < whole1) || v < sink1);
            uint8_t* unit = ring + slot * 2 * U;
            float s[2][NT][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) scores<D, NT>(unit + k * U, qf, qx, s[k]);
            if (!whole) {
                const int j0 = seq.pair(v) * kPair;
#pragma unroll
                for (int k = 0; k < 2; ++k) hide<D, NT>(unit + k * U, j0 + k * kTok, have >> k & 1u, pos, a, s[k]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");      // before the slot's next copy
                __syncwarp();
            }
            raise<D, NT, 2>(s, a, st);
#pragma unroll
            for (int k = 0; k < 2; ++k) add_values<D, NT>(unit + k * U, s[k], a, st);
            __syncwarp();       // every lane has read the slot: the unit kSlots further on goes there
            if (issued < n && ok) issue(issued++, slot);
            if (++slot == kSlots) {
                slot = 0;
                phase ^= 1u;
            }
        }
        // ---- join the warps
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = st.l[t][c];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (g == 0) {
                    sm.m[warp][8 * t + 2 * q + c] = st.m[t][c];
                    sm.l[warp][8 * t + 2 * q + c] = l;
                }
            }
        __syncthreads();
        if (threadIdx.x < kRows) {      // each warp's factor of a row, in place of its maximum; the row's sum
            const int r = threadIdx.x;
            float top = kNothing, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.m[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2((sm.m[w][r] - top) * a.scale);
                l += f * sm.l[w][r];
                sm.m[w][r] = f;
            }
            sm.top[r] = top;
            sm.l[0][r] = l;
        }
        float* wo = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    wo[(8 * t + 2 * q + (c & 1)) * S::kPitch + 16 * i + g + 8 * (c >> 1)] = st.o[t][i][c];
        __syncthreads();
        const bool begins = v0 == 0, ends = c1 == seq.cost();
        if (!kDirect && begins) {
            // its other pieces are the next ranges' first ones
            const int pieces = ends ? 1 : 1 + int((seq.cost() - c1 + quota - 1) / quota);
            cut = Desc{b, h, ht % a.RT, pieces, int(blockIdx.x), rows};
            if (a.by_segment && threadIdx.x == 0) a.desc[b * per_seq + ht] = cut;
        }
        float* part = a.part + (int64_t(blockIdx.x) * 2 + (begins ? 1 : 0)) * part_floats<D, NT>();
        for (int i = threadIdx.x; i < kRows * D / 4; i += kThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            if (r0 + r >= rows) break;
            float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm.m[w][r];
                const float4 v = *reinterpret_cast<const float4*>(sm.ring[w] + (r * S::kPitch + d) * 4);
                o[0] += f * v.x, o[1] += f * v.y, o[2] += f * v.z, o[3] += f * v.w;
            }
            const float l = sm.l[0][r];
            if (kDirect || (begins && ends)) {
                if (l == 0.f) o[0] = o[1] = o[2] = o[3] = 0.f;
                const float by = l == 0.f ? 1.f : l;
                *reinterpret_cast<uint2*>(a.o + row_at(r0 + r) + d) = make_uint2(pack_h2(o[0] / by, o[1] / by), pack_h2(o[2] / by, o[3] / by));
            } else {
                *reinterpret_cast<float4*>(part + r * (D + 4) + d) = make_float4(o[0], o[1], o[2], o[3]);
                if (d == 0) *reinterpret_cast<float2*>(part + r * (D + 4) + D) = make_float2(sm.top[r], l);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the rings' next copies follow these accesses
        __syncthreads();
        }
        left -= c1 - c0;
        c0 = 0;
        if (++ht == per_seq && left > 0) {
            ht = 0;
            seq = seq_of(a, ++b);
        }
    }
    if (!kDirect && !a.by_segment && threadIdx.x == 0) a.desc[blockIdx.x] = cut;     // of the last segment begun: the only one that can go on
    if (!ok) {
        // a wait ran out: give the copies under way their time to land before the CTA ends
        for (int i = 0; i < kSlots; ++i) mbar_wait_for(&full[i], phase ^ (i < int(slot)), kWaitLimitCycles / 16);
        if (a.status) atomicOr(a.status, kStatusTimeout);
    }
}

// Joins the pieces of the (sequence, head, tile)s that ranges cut: a CTA per row of one, kJoin / D pieces at a time, each thread
// with a running maximum of its own, so that all it needs of four pieces is loaded at once.
constexpr int kJoin = 512;

template <int D, int NT>
__global__ void __launch_bounds__(kJoin) join_kernel(const Args a) {
    constexpr int kRows = 8 * NT, stride = D + 4, kPar = kJoin / D, kBatch = 4;
    __shared__ float sm_m[kPar], sm_l[kPar], sm_o[kPar][D];
    grid_launch_dependents();
    grid_dependency_wait();
    const Desc ds = a.desc[blockIdx.x];
    const int r = blockIdx.y, R = ds.rt * kRows + r;
    if (ds.pieces < 2 || R >= ds.rows) return;
    // piece 0 begins the segment in its CTA's range; the others continue it in the CTAs after
    const int64_t size = part_floats<D, NT>();
    const float* base = a.part + int64_t(ds.cta) * 2 * size + r * stride;
    const int d = threadIdx.x % D, part = threadIdx.x / D;
    float m = kNothing, l = 0.f, o = 0.f;
    for (int p0 = part; p0 < ds.pieces; p0 += kBatch * kPar) {
        float pm[kBatch], pl[kBatch], po[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int p = p0 + i * kPar;
            const float* from = base + (p == 0 ? size : 2 * size * p);
            const bool there = p < ds.pieces;
            pm[i] = there ? from[D] : kNothing;
            pl[i] = there ? from[D + 1] : 0.f;
            po[i] = there ? from[d] : 0.f;
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) top = fmaxf(top, pm[i]);
        const float f = ex2((m - top) * a.scale);
        l *= f;
        o *= f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float e = ex2((pm[i] - top) * a.scale);
            l += e * pl[i];
            o += e * po[i];
        }
        m = top;
    }
    sm_o[part][d] = o;
    if (d == 0) {
        sm_m[part] = m;
        sm_l[part] = l;
    }
    __syncthreads();
    if (part) return;
    float top = kNothing;
#pragma unroll
    for (int i = 0; i < kPar; ++i) top = fmaxf(top, sm_m[i]);
    l = o = 0.f;
#pragma unroll
    for (int i = 0; i < kPar; ++i) {
        const float e = ex2((sm_m[i] - top) * a.scale);
        l += e * sm_l[i];
        o += e * sm_o[i][d];
    }
    a.o[((int64_t(ds.b) * a.T + R / a.G) * a.heads + ds.h * a.G + R % a.G) * D + d] = __float2half_rn(l == 0.f ? 0.f : o / l);
}

// Rows per tile: 8, or 16 where a kv head has more (the cache is then read half as often).
int tiles_of(int64_t T, int64_t G) { return T * G > 8 ? 2 : 1; }
int ctas_of(int D, int nt) { return sm_count() * resident(D, nt, 0); }

// Whether no segment can be long: the most units that one can have, by the table's width and the window. Up to kDirectUnits
// of them a CTA per segment is through sooner than the even split with its second kernel.
bool direct_of(int64_t width, int per_page, int window, int sinks, int64_t T, int64_t segments) {
    int64_t most = (width * per_page + 1) / 2;
    if (window > 0) most = std::min(most, (int64_t(sinks) + kPair - 1) / kPair + (window + T + kPair - 2) / kPair + 1);
    return most <= kDirectUnits && segments <= 0x7fffffff;
}

int64_t row_tiles(int64_t T, int64_t G) { return (T * G + 8 * tiles_of(T, G) - 1) / (8 * tiles_of(T, G)); }
int at_most_int(int64_t v) { return int(std::min<int64_t>(v, 0x7fffffff)); }

size_t workspace_of(const tern_cache* c, int64_t T, int64_t heads) {
    const int nt = tiles_of(T, heads / c->kv_heads);
    const size_t n = size_t(ctas_of(c->head_dim, nt));
    const size_t desc = (n * sizeof(Desc) + 255) & ~size_t(255);
    return (desc + n * 2 * size_t(8 * nt * (c->head_dim + 4)) * 4 + 255) & ~size_t(255);
}

template <int D, int NT, int kDirect>
bool configure() {
    static std::mutex mu;
    static bool configured[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev])
        configured[dev] = cudaFuncSetAttribute(attention_kernel<D, NT, kDirect>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(sizeof(Smem<D, NT, kDirect ? kDirect : kSplitWarps>))) == cudaSuccess;
    return configured[dev];
}

template <int D, int NT, int kWarps>
tern_status launch_direct(cudaLaunchConfig_t& cfg, const Args& a, int64_t segments) {
    if (!configure<D, NT, kWarps>()) return TERN_ERR_CUDA;
    cfg.gridDim = dim3(unsigned(segments), 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = sizeof(Smem<D, NT, kWarps>);
    return cudaLaunchKernelEx(&cfg, attention_kernel<D, NT, kWarps>, a) == cudaSuccess ? TERN_OK : TERN_ERR_CUDA;
}

template <int D, int NT>
tern_status launch(Args& a, void* workspace, cudaStream_t stream) {
    const int n = ctas_of(D, NT);
    a.RT = int(row_tiles(a.T, a.G));
    a.setup = setup_of(NT);
    a.desc = static_cast<Desc*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ((size_t(n) * sizeof(Desc) + 255) & ~size_t(255)));
    a.status = async_status_word();
    const int64_t segments = int64_t(a.B) * a.pool.heads * a.RT;
    a.by_segment = segments <= n;
    a.ndesc = a.by_segment ? int(segments) : n;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (direct_of(a.pool.width, a.pool.per_page, a.window, a.sinks, a.T, segments)) {
        if constexpr (NT == 1)      // (16 rows need the registers of 8 warps)
            if (segments <= sm_count()) return launch_direct<D, NT, kManyWarps>(cfg, a, segments);
        return launch_direct<D, NT, kFewWarps>(cfg, a, segments);
    }
    if (!configure<D, NT, 0>()) return TERN_ERR_CUDA;
    cfg.gridDim = dim3(unsigned(n), 1, 1);
    cfg.blockDim = dim3(kSplitWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = sizeof(Smem<D, NT, kSplitWarps>);
    if (cudaLaunchKernelEx(&cfg, attention_kernel<D, NT, 0>, a) != cudaSuccess) return TERN_ERR_CUDA;
    cfg.gridDim = dim3(unsigned(a.ndesc), unsigned(a.T * a.G < 8 * NT ? a.T * a.G : 8 * NT), 1);
    cfg.blockDim = dim3(kJoin, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, NT>, a) == cudaSuccess ? TERN_OK : TERN_ERR_CUDA;
}

tern_status check_attention(const tern_cache* c, int64_t B, int64_t T, int64_t heads, int64_t width, int64_t window, int64_t sinks) {
    const tern_status st = check_cache(c);
    if (st != TERN_OK) return st;
    if (!batch_ok(B, T, width) || T > 64 || heads <= 0 || heads % c->kv_heads || heads > 65535 || window < 0 || sinks < 0)
        return TERN_ERR_SHAPE;
    return TERN_OK;
}

}  // namespace
}  // namespace tern

using namespace tern;
using namespace tern::kv;

extern "C" size_t tern_cache_attention_workspace_bytes(const tern_cache* cache, int64_t B, int64_t T, int64_t heads,
                                                       int64_t width, int64_t window, int64_t sinks) {
    if (check_attention(cache, B, T, heads, width, window, sinks) != TERN_OK || B == 0 || T == 0) return 0;
    const int64_t segments = B * cache->kv_heads * row_tiles(T, heads / cache->kv_heads);
    if (direct_of(width, cache->page / kTok, at_most_int(window), at_most_int(sinks), T, segments)) return 0;
    return workspace_of(cache, T, heads);
}

extern "C" tern_status tern_cache_attention(const tern_cache* cache, const tern_half* q, int64_t B, int64_t T,
                                            int64_t heads, const int32_t* table, int64_t width, const int32_t* lens,
                                            const int32_t* counts, float scale, int64_t window, int64_t sinks,
                                            tern_half* o, void* workspace, size_t workspace_bytes, tern_stream stream) {
    const tern_status st = check_attention(cache, B, T, heads, width, window, sinks);
    if (st != TERN_OK) return st;
    if (!(fabsf(scale) <= kMaxScale)) return TERN_ERR_SHAPE;
    if (B == 0 || T == 0) return TERN_OK;
    if (!q || !o || !lens || (!table && width)) return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(o)) return TERN_ERR_ALIGN;
    const size_t bytes = size_t(B) * size_t(T) * size_t(heads) * size_t(cache->head_dim) * 2;
    if (overlaps(q, bytes, o, bytes)) return TERN_ERR_SHAPE;
    const size_t need = tern_cache_attention_workspace_bytes(cache, B, T, heads, width, window, sinks);
    if (need && (!workspace || workspace_bytes < need)) return TERN_ERR_WORKSPACE;
    if (workspace && !aligned16(workspace)) return TERN_ERR_ALIGN;
    Args a{};
    a.pool = pool_of(cache, table, width);
    a.q = reinterpret_cast<const __half*>(q);
    a.o = reinterpret_cast<__half*>(o);
    a.lens = lens;
    a.counts = counts;
    a.window = at_most_int(window);
    a.sinks = at_most_int(sinks);
    a.B = int(B);
    a.T = int(T);
    a.heads = int(heads);
    a.G = int(heads / cache->kv_heads);
    a.scale = fmaxf(fabsf(scale) * kLog2e, 1e-30f);    // zero is as good as 1e-30
    a.slack = kSlack / a.scale;
    a.sign = scale < 0.f ? 0x80008000u : 0u;
    cudaStream_t cs = as_cuda(stream);
    if (tiles_of(T, a.G) == 1)
        return cache->head_dim == 64 ? launch<64, 1>(a, workspace, cs) : launch<128, 1>(a, workspace, cs);
    return cache->head_dim == 64 ? launch<64, 2>(a, workspace, cs) : launch<128, 2>(a, workspace, cs);
}
