// The 4-bit KV cache: quantising new keys and values into pages, and reading them back.
//
// Per 64 entries of a head: s = rn16((max - min) / 15), z = rn16(min), c = rint((x - z) / s). Bound by HBM (a call moves each
// value once as fp16 and once in 4 bits), for long prompts about as much by the instructions of the quantising.
//
// One warp takes K or V of the 16 tokens of a block and kv head that are new (or asked for): lane 4 g + q holds, of tokens g and
// g + 8, entries 32 j + 8 q .. + 7, in 16-byte loads that read 64 consecutive bytes of a token per quad, and these
// eight codes are one word of the K layout: 512 consecutive bytes leave per warp and store. V's words hold two tokens of
// an entry: the eight lanes 8 q .. 8 q + 7 transpose their 8 x 8 codes (three exchanges), and lane 8 q + c then
// stores what belongs to lane 4 c + q. Where tokens of a block are not new, V's half words are stored one by one.
// Measured: append and read back of 4 x 4000 tokens, 8 heads of 128, 35 us of 147 MB (4.2 TB/s), the append alone 20.5 (it issues in
// 68 % of the slots; heads of 128 spill 8 bytes at 64 registers); one token of 64 sequences 8 us, two launches of latency.
#include "tern_cache.cuh"

namespace tern {
namespace {

using namespace kv;

constexpr int kThreads = 256;

struct Args {
    Pool pool;
    const int32_t* start;
    const int32_t* counts;
    int64_t B, T;
    int64_t blocks;         // of 16 tokens that T tokens can touch
};

// The warp's block of a call: K (kv = 0) or V of tokens pos0 + r, r < 16, of sequence b and kv head h; token t = off + r
// of the call.
struct Where {
    int64_t b, pos0, off;
    int h, kv;
};

__device__ __forceinline__ bool where(const Args& a, Where& w) {
    int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    w.h = int(i % a.pool.heads);
    i /= a.pool.heads;
    w.kv = int(i & 1);
    i >>= 1;
    const int64_t nth = i % a.blocks;
    w.b = i / a.blocks;
    if (w.b >= a.B) return false;
    const int64_t start = __ldg(a.start + w.b);
    w.pos0 = ((start >> 4) + nth) * kTok;      // (rounds down for a negative start too)
    w.off = w.pos0 - start;
    return w.off < a.T;
}

// 8 x 8 codes: lane r of eight holds row r (nibble c: column c); afterwards column r (nibble c: row c).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    const int lane = threadIdx.x & 31;
    uint32_t o = __shfl_xor_sync(0xffffffffu, v, 4);
    v = lane & 4 ? prmt(o, v, 0x7632) : prmt(v, o, 0x5410);                 // halves
    o = __shfl_xor_sync(0xffffffffu, v, 2);
    v = lane & 2 ? prmt(o, v, 0x7351) : prmt(v, o, 0x6240);                 // bytes
    o = __shfl_xor_sync(0xffffffffu, v, 1);
    return lane & 1 ? (v & 0xF0F0F0F0u) | (o >> 4 & 0x0F0F0F0Fu) : (v & 0x0F0F0F0Fu) | (o & 0x0F0F0F0Fu) << 4;
}

// The plain nibble order to that of a word of eight neighbouring columns (i at i / 2 + 4 (i % 2)).
__device__ __forceinline__ uint32_t pair_order(uint32_t w) {
    uint32_t lo = w & 0x0F0F0F0Fu, hi = w >> 4 & 0x0F0F0F0Fu;
    lo = (lo | lo >> 4) & 0x00FF00FFu, hi = (hi | hi >> 4) & 0x00FF00FFu;
    lo = (lo | lo >> 8) & 0x0000FFFFu, hi = (hi | hi >> 8) & 0x0000FFFFu;
    return lo | hi << 16;
}

template <int W>
__device__ __forceinline__ void store_words(uint32_t* to, const uint32_t (&w)[W]) {
    if constexpr (W == 4) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
}

template <int W>
__device__ __forceinline__ void fetch_words(const uint32_t* from, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(from);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(from);
        w[0] = v.x, w[1] = v.y;
    }
}

// The lane's entries of a token in codes (kPlain: in the plain order), their steps and zeros.
template <int D, bool kPlain>
__device__ __forceinline__ void quantise(const uint4 (&x)[D / 32], uint32_t (&w)[D / 32], __half (&s)[D / kGrp], __half (&z)[D / kGrp]) {
#pragma unroll
    for (int n = 0; n < D / kGrp; ++n) {
        __half2 lo2 = as_h2(x[2 * n].x), hi2 = lo2;
        take_range(x[2 * n], lo2, hi2);
        take_range(x[2 * n + 1], lo2, hi2);
        const float2 r = whole_range<4>(lo2, hi2);
        const float wide = __fsub_rn(r.y, r.x);
        s[n] = wide < INFINITY ? __float2half_rn(divided<15>(wide)) : __ushort_as_half(0x7FFFu);   // (a NaN or an infinity among them)
        z[n] = __float2half_rn(r.x);
        const float sf = __half2float(s[n]), zf = __half2float(z[n]), inv = reciprocal(sf);
#pragma unroll
        for (int j = 2 * n; j < 2 * n + 2; ++j) w[j] = sf > 0.f ? codes_of<0, kPlain>(x[j], zf, sf, inv) : 0u;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const Args a, const __half* __restrict__ k,
                                                          const __half* __restrict__ v) {
    constexpr int W = D / 32, NG = D / kGrp;
    grid_launch_dependents();
    grid_dependency_wait();
    Where w;
    if (!where(a, w)) return;
    const int64_t end = a.counts ? min(int64_t(__ldg(a.counts + w.b)), a.T) : a.T;     // tokens of the call
    if (w.off >= end || w.pos0 < 0) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const bool whole = w.off >= 0 && w.off + kTok <= end;
    const int64_t from = ((w.b * a.T + w.off) * a.pool.heads + w.h) * D, row = int64_t(a.pool.heads) * D;
    const __half* src = (w.kv ? v : k) + from;
    bool mine[2], some[2];
    uint4 x[2][W];              // the lane's two tokens, all loads under way at once
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t t = w.off + 8 * h + g;
        mine[h] = t >= 0 && t < end;
        some[h] = w.off + 8 * h + 7 >= 0 && w.off + 8 * h < end;
#pragma unroll
        for (int j = 0; j < W; ++j)
            x[h][j] = mine[h] ? __ldg(reinterpret_cast<const uint4*>(src + (8 * h + g) * row + 32 * j + 8 * q)) : make_uint4(0, 0, 0, 0);
    }
    uint8_t* unit = a.pool.block<D>(w.b, w.h, w.pos0 / kTok);
    if (!unit) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!some[h]) continue;             // (the whole warp)
        uint32_t c[W];
        __half s[NG], z[NG];
        if (!w.kv) {
            quantise<D, false>(x[h], c, s, z);
            if (mine[h]) store_words<W>(reinterpret_cast<uint32_t*>(unit) + (h * 32 + lane) * W, c);
        } else {
            quantise<D, true>(x[h], c, s, z);
#pragma unroll
            for (int j = 0; j < W; ++j) c[j] = transpose8(c[j]);
            // tokens 2 q' (low halves) and 2 q' + 1 (high) of q' = lane / 8, for the layout's lane 4 (lane % 8) + q'
            uint32_t* to = reinterpret_cast<uint32_t*>(unit + v_codes(D)) + (h * 32 + 4 * (lane & 7) + (lane >> 3)) * W;
            if (whole) {
                store_words<W>(to, c);
            } else {
                const int64_t t = w.off + 8 * h + 2 * (lane >> 3);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    if (t >= 0 && t < end) reinterpret_cast<uint16_t*>(to + j)[0] = uint16_t(c[j]);
                    if (t + 1 >= 0 && t + 1 < end) reinterpret_cast<uint16_t*>(to + j)[1] = uint16_t(c[j] >> 16);
                }
            }
        }
        if (mine[h] && q < NG) {
            const __half sq = NG == 1 || q == 0 ? s[0] : s[NG - 1], zq = NG == 1 || q == 0 ? z[0] : z[NG - 1];
            if (!w.kv) {
                reinterpret_cast<__half2*>(unit + k_scales(D))[(8 * h + g) * NG + q] = __halves2half2(sq, zq);
            } else {
                __half* at = reinterpret_cast<__half*>(unit + v_scales(D)) + ((g >> 1) * NG + q) * 8 + 2 * h + (g & 1);
                at[0] = sq;
                at[4] = zq;
            }
        }
    }
}

// Eight codes (a word of eight neighbouring columns) as fp16 values z + s c.
__device__ __forceinline__ uint4 values(uint32_t w, __half2 s, __half2 z) {
    const uint32_t w8 = w >> 8;
    return make_uint4(as_u32(__hfma2(as_h2(code_pair<0, 0>(w, w8)), s, z)), as_u32(__hfma2(as_h2(code_pair<1, 0>(w, w8)), s, z)),
                      as_u32(__hfma2(as_h2(code_pair<2, 0>(w, w8)), s, z)), as_u32(__hfma2(as_h2(code_pair<3, 0>(w, w8)), s, z)));
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const Args a, __half* __restrict__ k, __half* __restrict__ v) {
    constexpr int W = D / 32, NG = D / kGrp;
    grid_launch_dependents();
    grid_dependency_wait();
    Where w;
    if (!where(a, w)) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int64_t end = a.counts ? min(int64_t(__ldg(a.counts + w.b)), a.T) : a.T;
    const uint8_t* unit = w.pos0 >= 0 && w.off < end ? a.pool.block<D>(w.b, w.h, w.pos0 / kTok) : nullptr;
    const int64_t row = int64_t(a.pool.heads) * D;
    __half* to = (w.kv ? v : k) + ((w.b * a.T + w.off) * a.pool.heads + w.h) * D;
    uint32_t c[2][W] = {};
    __half2 s[2][NG], z[2][NG];
    if (unit) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int place = w.kv ? 4 * (lane & 7) + (lane >> 3) : lane;      // as append stored them
            fetch_words<W>(reinterpret_cast<const uint32_t*>(unit + (w.kv ? v_codes(D) : 0)) + (h * 32 + place) * W, c[h]);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const __half* at = w.kv ? reinterpret_cast<const __half*>(unit + v_scales(D)) + ((g >> 1) * NG + n) * 8 + 2 * h + (g & 1)
                                        : reinterpret_cast<const __half*>(unit + k_scales(D)) + ((8 * h + g) * NG + n) * 2;
                s[h][n] = __half2half2(at[0]);
                z[h][n] = __half2half2(at[w.kv ? 4 : 1]);
            }
        }
        if (w.kv) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < W; ++j) c[h][j] = pair_order(transpose8(c[h][j]));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t t = w.off + 8 * h + g;
        if (t < 0 || t >= a.T) continue;
        const bool there = unit && t < end;
#pragma unroll
        for (int j = 0; j < W; ++j)
            *reinterpret_cast<uint4*>(to + (8 * h + g) * row + 32 * j + 8 * q) =
                there ? values(c[h][j], s[h][j / 2], z[h][j / 2]) : make_uint4(0, 0, 0, 0);
    }
}

tern_status check_call(const tern_cache* c, const void* k, const void* v, int64_t B, int64_t T, const int32_t* table,
                       int64_t width, const int32_t* start) {
    const tern_status st = check_cache(c);
    if (st != TERN_OK) return st;
    if (!batch_ok(B, T, width)) return TERN_ERR_SHAPE;
    if (B == 0 || T == 0) return TERN_OK;
    if (!k || !v || (!table && width) || !start) return TERN_ERR_NULL;
    return aligned16(k) && aligned16(v) ? TERN_OK : TERN_ERR_ALIGN;
}

int64_t blocks_of(int64_t T) { return (T + kTok - 2) / kTok + 1; }

bool grid_for(const tern_cache* c, int64_t B, int64_t T, unsigned& n) {
    const int64_t ctas = (B * blocks_of(T) * 2 * c->kv_heads * 32 + kThreads - 1) / kThreads;
    n = unsigned(ctas);
    return ctas <= 0x7fffffff;
}

}  // namespace
}  // namespace tern

using namespace tern;
using namespace tern::kv;

extern "C" tern_status tern_cache_append(const tern_cache* cache, const tern_half* k, const tern_half* v, int64_t B,
                                         int64_t T, const int32_t* table, int64_t width, const int32_t* start,
                                         const int32_t* counts, tern_stream stream) {
    const tern_status st = check_call(cache, k, v, B, T, table, width, start);
    if (st != TERN_OK || B == 0 || T == 0) return st;
    unsigned n;
    if (!grid_for(cache, B, T, n)) return TERN_ERR_SHAPE;
    const Args a{pool_of(cache, table, width), start, counts, B, T, blocks_of(T)};
    auto kernel = cache->head_dim == 64 ? append_kernel<64> : append_kernel<128>;
    return launch_dependent(kernel, n, kThreads, as_cuda(stream), a, reinterpret_cast<const __half*>(k), reinterpret_cast<const __half*>(v));
}

extern "C" tern_status tern_cache_read(const tern_cache* cache, tern_half* k, tern_half* v, int64_t B, int64_t T,
                                       const int32_t* table, int64_t width, const int32_t* start,
                                       const int32_t* counts, tern_stream stream) {
    const tern_status st = check_call(cache, k, v, B, T, table, width, start);
    if (st != TERN_OK || B == 0 || T == 0) return st;
    unsigned n;
    if (!grid_for(cache, B, T, n)) return TERN_ERR_SHAPE;
    const Args a{pool_of(cache, table, width), start, counts, B, T, blocks_of(T)};
    auto kernel = cache->head_dim == 64 ? read_kernel<64> : read_kernel<128>;
    return launch_dependent(kernel, n, kThreads, as_cuda(stream), a, reinterpret_cast<__half*>(k), reinterpret_cast<__half*>(v));
}
