// The 4-bit KV cache: quantising new keys and values into pages, and reading them back.
//
// Per 64 entries of a head: s = rn16((max - min) / 15), z = rn16(min), c = rint((x - z) / s). One warp takes a token of
// one kv head: lane i holds entries (D / 32) i .. , the range is taken over the lanes of a group, and the
// codes go to their places in the block of 16 tokens (tern.h).
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
};

// The warp's token t of sequence b and head h, with its place: false past the batch.
__device__ __forceinline__ bool token_of(const Args& a, int64_t& b, int64_t& t, int& h) {
    int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    h = int(i % a.pool.heads);
    i /= a.pool.heads;
    t = i % a.T;
    b = i / a.T;
    return b < a.B;
}

template <int D>
__device__ __forceinline__ void quantise_to(const __half* __restrict__ src, uint8_t* unit, int r, bool is_v) {
    constexpr int E = D / 32;            // entries of a lane
    const int lane = threadIdx.x & 31;
    float f[E];
    float lo = INFINITY, hi = -INFINITY;
    bool odd = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        f[e] = __half2float(src[lane * E + e]);
        lo = fminf(lo, f[e]);
        hi = fmaxf(hi, f[e]);
        odd |= !(fabsf(f[e]) < INFINITY);
    }
#pragma unroll
    for (int o = 1; o < kGrp / E; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        odd |= __shfl_xor_sync(0xffffffffu, int(odd), o) != 0;
    }
    __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const __half zh = __float2half_rn(lo);
    if (odd) sh = __ushort_as_half(0x7FFFu);
    const float s = __half2float(sh), z = __half2float(zh), inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
    uint32_t c[E];
#pragma unroll
    for (int e = 0; e < E; ++e) c[e] = s > 0.f ? uint32_t(code_of(f[e], z, s, inv, 0)) : 0u;
    const int grp = lane * E / kGrp;
    if (!is_v) {
        // words of 8 entries: column i at nibble i / 2 + 4 (i % 2); 8 / E lanes share a word
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = (lane * E + e) & 7;
            w |= c[e] << (4 * (i / 2 + 4 * (i & 1)));
        }
#pragma unroll
        for (int o = 1; o < 8 / E; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
        if ((lane * E) % 8 == 0) {
            const int j = lane * E / 32, q = lane * E / 8 % 4;
            reinterpret_cast<uint32_t*>(unit)[(r * 4 + q) * (D / 32) + j] = w;
        }
        if ((lane * E) % kGrp == 0) {
            __half* at = reinterpret_cast<__half*>(unit + k_scales(D)) + (r * (D / kGrp) + grp) * 2;
            at[0] = sh;
            at[1] = zh;
        }
    } else {
        // entry d of word (h, g = d % 8, q, j = d / 32): nibble 2 (d / 16 % 2) + d / 8 % 2 of the token's half word. The lane
        // with entry d < 8 of a 32 gathers the other three.
        const int h = r >> 3, q = (r & 7) >> 1, odd_tok = r & 1;
        uint16_t* out = reinterpret_cast<uint16_t*>(unit + v_codes(D));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = lane * E + e;
            uint32_t w = c[e] << (4 * (d / 8 % 4 / 2 * 2 + d / 8 % 2));
            w |= __shfl_xor_sync(0xffffffffu, w, 8 / E);
            w |= __shfl_xor_sync(0xffffffffu, w, 16 / E);
            if (d % 32 < 8) out[(((h * 8 + d % 8) * 4 + q) * (D / 32) + d / 32) * 2 + odd_tok] = uint16_t(w);
        }
        if ((lane * E) % kGrp == 0) {
            __half* at = reinterpret_cast<__half*>(unit + v_scales(D)) + (q * (D / kGrp) + grp) * 8 + 2 * h + odd_tok;
            at[0] = sh;
            at[4] = zh;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const Args a, const __half* __restrict__ k,
                                                          const __half* __restrict__ v) {
    int64_t b, t;
    int h;
    if (!token_of(a, b, t, h)) return;
    if (a.counts && t >= __ldg(a.counts + b)) return;
    const int64_t at = int64_t(__ldg(a.start + b)) + t;
    uint8_t* unit = at < 0 ? nullptr : a.pool.block<D>(b, h, at / kTok);
    if (!unit) return;
    const int64_t from = ((b * a.T + t) * a.pool.heads + h) * D;
    quantise_to<D>(k + from, unit, int(at % kTok), false);
    quantise_to<D>(v + from, unit, int(at % kTok), true);
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const Args a, __half* __restrict__ k, __half* __restrict__ v) {
    constexpr int E = D / 32;
    int64_t b, t;
    int h;
    if (!token_of(a, b, t, h)) return;
    const int lane = threadIdx.x & 31;
    const int64_t at = int64_t(__ldg(a.start + b)) + t, to = ((b * a.T + t) * a.pool.heads + h) * D + lane * E;
    const bool wanted = at >= 0 && !(a.counts && t >= __ldg(a.counts + b));
    const uint8_t* unit = wanted ? a.pool.block<D>(b, h, at / kTok) : nullptr;
    const int r = int(at % kTok), grp = lane * E / kGrp;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float ko = 0.f, vo = 0.f;
        if (unit) {
            const int d = lane * E + e, i = d & 7;
            const __half* ks = reinterpret_cast<const __half*>(unit + k_scales(D)) + (r * (D / kGrp) + grp) * 2;
            const uint32_t kw = reinterpret_cast<const uint32_t*>(unit)[(r * 4 + d / 8 % 4) * (D / 32) + d / 32];
            ko = __half2float(ks[1]) + __half2float(ks[0]) * float(kw >> (4 * (i / 2 + 4 * (i & 1))) & 15u);
            const int hh = r >> 3, q = (r & 7) >> 1, odd = r & 1;
            const __half* vs = reinterpret_cast<const __half*>(unit + v_scales(D)) + (q * (D / kGrp) + grp) * 8 + 2 * hh + odd;
            const uint32_t vw = reinterpret_cast<const uint32_t*>(unit + v_codes(D))[((hh * 8 + d % 8) * 4 + q) * (D / 32) + d / 32];
            vo = __half2float(vs[4]) + __half2float(vs[0]) * float(vw >> (4 * (d / 16 % 2 * 2 + d / 8 % 2) + 16 * odd) & 15u);
        }
        k[to + e] = __float2half_rn(ko);
        v[to + e] = __float2half_rn(vo);
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

bool grid_for(const tern_cache* c, int64_t B, int64_t T, unsigned& n) {
    const int64_t blocks = (B * T * c->kv_heads * 32 + kThreads - 1) / kThreads;
    n = unsigned(blocks);
    return blocks <= 0x7fffffff;
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
    const Args a{pool_of(cache, table, width), start, counts, B, T};
    auto kernel = cache->head_dim == 64 ? append_kernel<64> : append_kernel<128>;
    kernel<<<n, kThreads, 0, as_cuda(stream)>>>(a, reinterpret_cast<const __half*>(k), reinterpret_cast<const __half*>(v));
    return launched();
}

extern "C" tern_status tern_cache_read(const tern_cache* cache, tern_half* k, tern_half* v, int64_t B, int64_t T,
                                       const int32_t* table, int64_t width, const int32_t* start,
                                       const int32_t* counts, tern_stream stream) {
    const tern_status st = check_call(cache, k, v, B, T, table, width, start);
    if (st != TERN_OK || B == 0 || T == 0) return st;
    unsigned n;
    if (!grid_for(cache, B, T, n)) return TERN_ERR_SHAPE;
    const Args a{pool_of(cache, table, width), start, counts, B, T};
    auto kernel = cache->head_dim == 64 ? read_kernel<64> : read_kernel<128>;
    kernel<<<n, kThreads, 0, as_cuda(stream)>>>(a, reinterpret_cast<__half*>(k), reinterpret_cast<__half*>(v));
    return launched();
}
