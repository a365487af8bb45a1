// Attention of a sequence's last tokens over its 4-bit KV cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q k_j - max),  k_j = z + s c (per 64 entries), v_j likewise.
//
// The queries that share a kv head (heads / kv_heads of them for each of the T tokens) are the rows, in tiles
// of 8. A warp takes blocks of 16 cached tokens and runs both products on mma.sync m16n8k16 with the rows as
// the instruction's 8 columns:
//   S^T [16 tokens, 8 rows] = C_K [16 tokens, D] Q^T, one accumulator per 64 entries, then s (.) + z sum(q) in fp32;
//   O^T [D, 8 rows] += V^T [D, 16 tokens] P^T [16 tokens, 8 rows].
// The cache's layout is that of the A operands, so codes go from memory to the instruction with no shuffle: a
// word is four pairs (entries of a token for K, two tokens of an entry for V). P^T is S^T's
// fragment transposed within the warp (movmatrix). Every warp keeps its own running maximum, sum and O^T; a
// block's warps join theirs in shared memory at the end.
#include <math.h>

#include "tern_cache.cuh"

namespace tern {
namespace {

using namespace kv;

constexpr int kWarps = 4;
constexpr int kRows = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    Pool pool;
    const __half* q;
    __half* o;
    const int32_t* lens;
    const int32_t* counts;
    int64_t window, sinks;
    int B, T, heads, G;         // G = heads per kv head
    float scale;
};

__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
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

// What a lane knows of its two rows (columns 2 q and 2 q + 1 of the tile): the token each query sits at (-1:
// no query).
struct Rows {
    int64_t pos[2];
    int64_t first, last;        // of the tile's queries: the smallest and the largest token
};

__device__ __forceinline__ bool sees(int64_t pos, int64_t j, int64_t window, int64_t sinks) {
    return j <= pos && (window <= 0 || j > pos - window || j < sinks);
}

template <int D>
struct State {
    float m[2], l[2];
    float o[D / 16][4];
};

template <int D>
__device__ __forceinline__ void init(State<D>& st) {
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
}

// One block of 16 tokens, j0 the first. kMask: some row does not see some token.
template <int D, bool kMask>
__device__ __forceinline__ void block_step(const uint8_t* unit, int64_t j0, const uint32_t (&qf)[D / 32][4],
                                           const float (&qsum)[D / kGrp][2], const Rows& rows, const Args& a,
                                           float scale, State<D>& st) {
    constexpr int W = D / 32, NG = D / kGrp;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    uint32_t ka[W], kb[W], va[W], vb[W];
    load_words(unit + lane * W * 4, ka);
    load_words(unit + (32 + lane) * W * 4, kb);
    load_words(unit + v_codes(D) + lane * W * 4, va);
    load_words(unit + v_codes(D) + (32 + lane) * W * 4, vb);

    float s[4] = {0.f, 0.f, 0.f, 0.f};   // [token g: rows 2q, 2q+1][token g + 8: the same]
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 2 * n; j < 2 * n + 2; ++j) {
            const uint32_t a8 = ka[j] >> 8, b8 = kb[j] >> 8;
            const uint32_t A0[4] = {code_pair<0, 0>(ka[j], a8), code_pair<0, 0>(kb[j], b8), code_pair<1, 0>(ka[j], a8),
                                    code_pair<1, 0>(kb[j], b8)};
            const uint32_t A1[4] = {code_pair<2, 0>(ka[j], a8), code_pair<2, 0>(kb[j], b8), code_pair<3, 0>(ka[j], a8),
                                    code_pair<3, 0>(kb[j], b8)};
            mma_16816(acc, A0, qf[j][0], qf[j][1]);
            mma_16816(acc, A1, qf[j][2], qf[j][3]);
        }
        const __half2* ks = reinterpret_cast<const __half2*>(unit + k_scales(D));
        const float2 s0 = __half22float2(ks[g * NG + n]), s1 = __half22float2(ks[(g + 8) * NG + n]);
        s[0] += s0.x * acc[0] + s0.y * qsum[n][0];
        s[1] += s0.x * acc[1] + s0.y * qsum[n][1];
        s[2] += s1.x * acc[2] + s1.y * qsum[n][0];
        s[3] += s1.x * acc[3] + s1.y * qsum[n][1];
    }
    // Steps and zeros of the lane's V tokens 2q, 2q + 1 (index 0) and 2q + 8, 2q + 9 (index 1), per 64 entries.
    uint32_t vs[NG][2], vz[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        const uint4 v = *reinterpret_cast<const uint4*>(unit + v_scales(D) + (q * NG + n) * 16);
        vs[n][0] = v.x, vs[n][1] = v.y, vz[n][0] = v.z, vz[n][1] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] *= scale;
    if (kMask) {
        // A V token that no row sees, or whose scales are not finite, counts as zeros in the product; a
        // row that sees one of the latter becomes NaN through its sum instead.
        const __half* vh = reinterpret_cast<const __half*>(unit + v_scales(D));
        bool odd[2] = {false, false};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float f = __half2float(vh[((g >> 1) * NG + n) * 8 + z * 4 + 2 * h + (g & 1)]);
                    odd[h] |= !(fabsf(f) < INFINITY);
                }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!sees(rows.pos[i & 1], j0 + g + 8 * (i >> 1), a.window, a.sinks)) s[i] = -INFINITY;
            else if (odd[i >> 1]) s[i] = NAN;
        }
        const bool used0 = s[0] != -INFINITY || s[1] != -INFINITY, used1 = s[2] != -INFINITY || s[3] != -INFINITY;
        unsigned keep0 = __ballot_sync(0xffffffffu, used0 && !odd[0]), keep1 = __ballot_sync(0xffffffffu, used1 && !odd[1]);
        // bits 4 t .. 4 t + 3: token t, any of its lanes
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const unsigned keep = h ? keep1 : keep0;
            const uint32_t mask = ((keep >> (8 * q)) & 0xFu ? 0x0000FFFFu : 0u) | ((keep >> (8 * q + 4)) & 0xFu ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                vs[n][h] &= mask;
                vz[n][h] &= mask;
            }
        }
    }
    // running maximum of each row: over the lane's two tokens, then over the 8 lanes of its column
    float mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
    }
    if (__any_sync(0xffffffffu, mx[0] > st.m[0] || mx[1] > st.m[1])) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float m = fmaxf(st.m[c], mx[c]);
            const float f = m > st.m[c] ? exp2f(st.m[c] - m) : 1.f;
            st.m[c] = m;
            st.l[c] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                st.o[i][c] *= f;
                st.o[i][2 + c] *= f;
            }
        }
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float m = st.m[i & 1];
        p[i] = exp2f(s[i] - (m == -INFINITY ? 0.f : m));
    }
    st.l[0] += p[0] + p[2];
    st.l[1] += p[1] + p[3];
    const uint32_t b0 = transposed(pack_h2(p[0], p[1])), b1 = transposed(pack_h2(p[2], p[3]));
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const uint32_t a8 = va[j] >> 8, b8 = vb[j] >> 8;
        const __half2 s0 = as_h2(vs[j / 2][0]), s1 = as_h2(vs[j / 2][1]), z0 = as_h2(vz[j / 2][0]), z1 = as_h2(vz[j / 2][1]);
        const uint32_t A0[4] = {as_u32(__hfma2(as_h2(code_pair<0, 0>(va[j], a8)), s0, z0)),
                                as_u32(__hfma2(as_h2(code_pair<1, 0>(va[j], a8)), s0, z0)),
                                as_u32(__hfma2(as_h2(code_pair<0, 0>(vb[j], b8)), s1, z1)),
                                as_u32(__hfma2(as_h2(code_pair<1, 0>(vb[j], b8)), s1, z1))};
        const uint32_t A1[4] = {as_u32(__hfma2(as_h2(code_pair<2, 0>(va[j], a8)), s0, z0)),
                                as_u32(__hfma2(as_h2(code_pair<3, 0>(va[j], a8)), s0, z0)),
                                as_u32(__hfma2(as_h2(code_pair<2, 0>(vb[j], b8)), s1, z1)),
                                as_u32(__hfma2(as_h2(code_pair<3, 0>(vb[j], b8)), s1, z1))};
        mma_16816(st.o[2 * j], A0, b0, b1);
        mma_16816(st.o[2 * j + 1], A1, b0, b1);
    }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const Args a) {
    constexpr int W = D / 32, NG = D / kGrp;
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows], sm_o[kWarps][kRows][D + 1];
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.z;
    const int h = blockIdx.y, r0 = blockIdx.x * kRows;
    const int64_t len = max(0, __ldg(a.lens + b));
    const int cnt = a.counts ? min(max(__ldg(a.counts + b), 0), a.T) : a.T;
    if (r0 >= cnt * a.G) return;
    // row R of the tile: query token R / G, head R % G of the kv head
    auto q_at = [&](int R) { return ((b * a.T + R / a.G) * a.heads + h * a.G + R % a.G) * D; };
    auto pos_of = [&](int R) { return R < cnt * a.G ? len - cnt + R / a.G : int64_t(-1); };

    uint32_t qf[W][4];
    float part[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) part[n] = 0.f;
    const bool real = r0 + g < cnt * a.G;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const uint4 v = real ? *reinterpret_cast<const uint4*>(a.q + q_at(r0 + g) + 32 * j + 8 * q) : make_uint4(0, 0, 0, 0);
        qf[j][0] = v.x, qf[j][1] = v.y, qf[j][2] = v.z, qf[j][3] = v.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(as_h2(qf[j][i]));
            part[j / 2] += f.x + f.y;
        }
    }
    float qsum[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        part[n] += __shfl_xor_sync(0xffffffffu, part[n], 1);
        part[n] += __shfl_xor_sync(0xffffffffu, part[n], 2);
        qsum[n][0] = __shfl_sync(0xffffffffu, part[n], 8 * q);
        qsum[n][1] = __shfl_sync(0xffffffffu, part[n], 8 * q + 4);
    }
    Rows rows;
    rows.pos[0] = pos_of(r0 + 2 * q);
    rows.pos[1] = pos_of(r0 + 2 * q + 1);
    rows.first = len - cnt + r0 / a.G;
    rows.last = len - cnt + (min(r0 + kRows, cnt * a.G) - 1) / a.G;
    const float scale = a.scale * kLog2e;

    State<D> st;
    init(st);
    const int64_t blocks = rows.last < 0 ? 0 : min(rows.last / kTok + 1, a.pool.width * a.pool.per_page);
    for (int64_t blk = warp; blk < blocks; blk += kWarps) {
        const int64_t j0 = blk * kTok;
        if (a.window > 0 && j0 + kTok - 1 <= rows.first - a.window && j0 >= a.sinks) continue;
        const uint8_t* unit = a.pool.block<D>(b, h, blk);
        if (!unit) continue;
        const bool whole = j0 + kTok - 1 <= rows.first && (a.window <= 0 || j0 > rows.last - a.window || j0 + kTok <= a.sinks);
        if (whole) block_step<D, false>(unit, j0, qf, qsum, rows, a, scale, st);
        else block_step<D, true>(unit, j0, qf, qsum, rows, a, scale, st);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], o);
        st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], o);
    }
    if (g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            sm_m[warp][2 * q + c] = st.m[c];
            sm_l[warp][2 * q + c] = st.l[c];
        }
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sm_o[warp][2 * q + (c & 1)][16 * i + g + 8 * (c >> 1)] = st.o[i][c];
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * D; i += kWarps * 32) {
        const int r = i / D, d = i % D;
        if (r0 + r >= cnt * a.G) continue;
        float m = -INFINITY;
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_m[w][r]);
        float l = 0.f, o = 0.f;
        for (int w = 0; w < kWarps; ++w) {
            const float f = m == -INFINITY ? 1.f : exp2f(sm_m[w][r] - m);
            l += f * sm_l[w][r];
            o += f * sm_o[w][r][d];
        }
        a.o[q_at(r0 + r) + d] = __float2half_rn(l == 0.f ? 0.f : o / l);
    }
}

tern_status check_attention(const tern_cache* c, int64_t B, int64_t T, int64_t heads) {
    const tern_status st = check_cache(c);
    if (st != TERN_OK) return st;
    if (!batch_ok(B, T, 0) || T > 64 || heads <= 0 || heads % c->kv_heads || heads > 65535) return TERN_ERR_SHAPE;
    return TERN_OK;
}

}  // namespace
}  // namespace tern

using namespace tern;
using namespace tern::kv;

extern "C" size_t tern_cache_attention_workspace_bytes(const tern_cache* cache, int64_t B, int64_t T, int64_t heads) {
    return 0;
}

extern "C" tern_status tern_cache_attention(const tern_cache* cache, const tern_half* q, int64_t B, int64_t T,
                                            int64_t heads, const int32_t* table, int64_t width, const int32_t* lens,
                                            const int32_t* counts, float scale, int64_t window, int64_t sinks,
                                            tern_half* o, void* workspace, size_t workspace_bytes, tern_stream stream) {
    const tern_status st = check_attention(cache, B, T, heads);
    if (st != TERN_OK) return st;
    if (!batch_ok(B, T, width) || window < 0 || sinks < 0 || !isfinite(scale)) return TERN_ERR_SHAPE;
    if (B == 0 || T == 0) return TERN_OK;
    if (!q || !o || !lens || (!table && width)) return TERN_ERR_NULL;
    if (!aligned16(q) || !aligned16(o)) return TERN_ERR_ALIGN;
    const size_t bytes = size_t(B) * size_t(T) * size_t(heads) * size_t(cache->head_dim) * 2;
    if (overlaps(q, bytes, o, bytes)) return TERN_ERR_SHAPE;
    const size_t need = tern_cache_attention_workspace_bytes(cache, B, T, heads);
    if (need && (!workspace || workspace_bytes < need)) return TERN_ERR_WORKSPACE;
    if (workspace && !aligned16(workspace)) return TERN_ERR_ALIGN;
    Args a{pool_of(cache, table, width), reinterpret_cast<const __half*>(q), reinterpret_cast<__half*>(o), lens, counts,
           window, sinks, int(B), int(T), int(heads), int(heads / cache->kv_heads), scale};
    const dim3 grid(unsigned((T * a.G + kRows - 1) / kRows), unsigned(cache->kv_heads), unsigned(B));
    auto kernel = cache->head_dim == 64 ? attention_kernel<64> : attention_kernel<128>;
    kernel<<<grid, kWarps * 32, 0, as_cuda(stream)>>>(a);
    return launched();
}
