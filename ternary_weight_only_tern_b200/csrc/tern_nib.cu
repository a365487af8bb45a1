// 4-bit weights: the fit of a dense W, the packing of another source's codes, and the way back to fp16.
//
// Per (row, group of 32, 64 or 128): step s and offset mu from the group's range, c = rint((w - mu) / s) + 8
// (tern.h has the formulas). Elementwise with a small reduction, so bound by HBM: a fit reads 2 N K bytes and
// writes N K / 2 and the scales.
//
// One warp takes 8 rows x 128 columns, half of a strip's block: lane 4 g + q holds row g's columns
// 32 j + 8 q .. + 7 (j = 0 .. 3), four 16-byte loads in which a quad reads 64 consecutive bytes of a row, and
// these are the four words that the layout gives the lane, so the codes leave as one 16-byte store per
// lane and 512 consecutive bytes per warp. A group's range is taken over the lane's registers and the quad.
// Measured: 4096 x 12288, group 64, fit and back to fp16 50 us of 257 MB (5.2 TB/s), 30 of them the fit, which issues in 76 % of the
// slots, most of it the quantising; packing, a synchronous call, 51 us.
#include "tern_nib.cuh"

namespace tern {
namespace {

using namespace nib;

constexpr int kThreads = 256;

struct Place {            // a warp's 8 rows x 128 columns, and the lane's part of it
    int64_t strip, kb;
    int h, g, q;
    int64_t row;
};

// Warps count columns fastest, then the strip's halves, so that neighbouring warps read on along the rows.
__device__ __forceinline__ bool place_of(int64_t strips, int64_t KB, Place& p) {
    const int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    p.kb = i % KB;
    p.h = int(i / KB & 1);
    p.strip = i / KB >> 1;
    p.g = lane >> 2;
    p.q = lane & 3;
    p.row = p.strip * 16 + p.h * 8 + p.g;
    return p.strip < strips;
}

__device__ __forceinline__ int64_t word_at(const Place& p, int64_t KB) {
    return ((p.strip * KB + p.kb) * kBlockWords) + ((p.h * 8 + p.g) * 4 + p.q) * 4;
}

// Element of scale and mu for the group that holds column 32 j of the block.
template <int kGrp>
__device__ __forceinline__ int64_t scale_at(const Place& p, int64_t KB, int j) {
    constexpr int per = kGroup / kGrp;
    return ((p.strip * KB + p.kb) * per + j * 32 / kGrp) * 16 + 2 * p.g + p.h;
}

template <int kGrp>
__global__ void __launch_bounds__(kThreads) fit_kernel(const __half* __restrict__ W, int64_t N, int64_t K, int offset,
                                                       uint32_t* __restrict__ codes, __half* __restrict__ scale,
                                                       __half* __restrict__ mu) {
    grid_dependency_wait();     // (and no early start for the kernel after: it may read these weights as static ones)
    const int64_t KB = K / kGroup;
    Place p;
    if (!place_of((N + 15) / 16, KB, p)) return;
    const bool real = p.row < N;
    uint4 raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        raw[j] = real ? __ldg(reinterpret_cast<const uint4*>(W + p.row * K + p.kb * kGroup + 32 * j + 8 * p.q))
                      : make_uint4(0, 0, 0, 0);
    constexpr int span = kGrp / 32;      // words of a lane that share a group
    uint32_t out[4];
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += span) {
        __half2 lo2 = as_h2(raw[j0].x), hi2 = lo2;
#pragma unroll
        for (int j = j0; j < j0 + span; ++j) take_range(raw[j], lo2, hi2);
        const float2 range = whole_range<4>(lo2, hi2);
        const float lo = range.x, hi = range.y;
        const float wide = offset ? __fsub_rn(hi, lo) : fmaxf(fabsf(lo), fabsf(hi));
        __half sh = __float2half_rn(offset ? divided<15>(wide) : divided<7>(wide));
        const __half mh = __float2half_rn(offset ? __fadd_rn(lo, __fmul_rn(8.f, __half2float(sh))) : 0.f);
        if (!(wide < INFINITY)) sh = __ushort_as_half(0x7FFFu);       // a NaN or an infinity in the group
        const float s = __half2float(sh), m = __half2float(mh), inv = reciprocal(s);
#pragma unroll
        for (int j = j0; j < j0 + span; ++j) out[j] = s > 0.f ? codes_of<8>(raw[j], m, s, inv) : 0x88888888u;
        if (p.q == 0) {
            const int64_t at = scale_at<kGrp>(p, KB, j0);
            scale[at] = sh;
            if (offset) mu[at] = mh;
        }
    }
    *reinterpret_cast<uint4*>(codes + word_at(p, KB)) = make_uint4(out[0], out[1], out[2], out[3]);
}

template <int kGrp>
__global__ void __launch_bounds__(kThreads) dequant_kernel(const uint32_t* __restrict__ codes,
                                                           const __half* __restrict__ scale,
                                                           const __half* __restrict__ mu, int64_t N, int64_t K,
                                                           __half* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t KB = K / kGroup;
    Place p;
    if (!place_of((N + 15) / 16, KB, p) || p.row >= N) return;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(codes + word_at(p, KB)));
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t at = scale_at<kGrp>(p, KB, j);
        const __half2 s = __half2half2(__ldg(scale + at));
        const __half2 m = __half2half2(mu ? __ldg(mu + at) : __float2half_rn(0.f));
        const uint32_t w = words[j], w8 = w >> 8;
        const uint4 o = make_uint4(as_u32(__hfma2(as_h2(code_pair<0, 8>(w, w8)), s, m)),
                                   as_u32(__hfma2(as_h2(code_pair<1, 8>(w, w8)), s, m)),
                                   as_u32(__hfma2(as_h2(code_pair<2, 8>(w, w8)), s, m)),
                                   as_u32(__hfma2(as_h2(code_pair<3, 8>(w, w8)), s, m)));
        *reinterpret_cast<uint4*>(out + p.row * K + p.kb * kGroup + 32 * j + 8 * p.q) = o;
    }
}

template <int kGrp>
__global__ void __launch_bounds__(kThreads) pack_kernel(const uint8_t* __restrict__ c, const __half* __restrict__ s,
                                                        const __half* __restrict__ m, int64_t N, int64_t K,
                                                        uint32_t* __restrict__ codes, __half* __restrict__ scale,
                                                        __half* __restrict__ mu, unsigned int* __restrict__ flag) {
    const int64_t KB = K / kGroup;
    Place p;
    if (!place_of((N + 15) / 16, KB, p)) return;
    const bool real = p.row < N;
    uint32_t out[4];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t col = p.kb * kGroup + 32 * j + 8 * p.q;
        const uint64_t v = real ? __ldg(reinterpret_cast<const unsigned long long*>(c + p.row * K + col))
                                : 0x0808080808080808ull;
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t n = uint32_t(v >> (8 * i)) & 0xFFu;
            bad |= n > 15u;
            n = n > 15u ? 15u : n;
            w |= n << (4 * (i / 2 + 4 * (i % 2)));
        }
        out[j] = w;
        if (p.q == 0 && j * 32 % kGrp == 0) {
            const int64_t at = scale_at<kGrp>(p, KB, j), from = p.row * (K / kGrp) + (p.kb * kGroup + 32 * j) / kGrp;
            scale[at] = real ? s[from] : __float2half_rn(0.f);
            if (mu) mu[at] = real ? m[from] : __float2half_rn(0.f);
        }
    }
    *reinterpret_cast<uint4*>(codes + word_at(p, KB)) = make_uint4(out[0], out[1], out[2], out[3]);
    if (bad) atomicOr(flag, 1u);
}

unsigned blocks_for(int64_t N, int64_t K) {
    return unsigned((((N + 15) / 16) * 2 * (K / kGroup) * 32 + kThreads - 1) / kThreads);
}

}  // namespace
}  // namespace tern

using namespace tern;
using namespace tern::nib;

extern "C" tern_status tern_nib_fit(const tern_half* W, int64_t N, int64_t K, int32_t group, int32_t offset,
                                    uint32_t* codes, tern_half* scale, tern_half* mu, tern_stream stream) {
    const tern_status st = check_shape(N, K, group);
    if (st != TERN_OK) return st;
    if (!W || !codes || !scale || (offset && !mu)) return TERN_ERR_NULL;
    if (!aligned16(W) || !aligned16(codes) || !aligned16(scale) || (offset && !aligned16(mu))) return TERN_ERR_ALIGN;
    auto kernel = group == 32 ? fit_kernel<32> : group == 64 ? fit_kernel<64> : fit_kernel<128>;
    return launch_dependent(kernel, blocks_for(N, K), kThreads, as_cuda(stream), reinterpret_cast<const __half*>(W), N, K, int(offset != 0),
                            codes, reinterpret_cast<__half*>(scale), reinterpret_cast<__half*>(mu));
}

extern "C" tern_status tern_nib_dequant(const tern_nib_weight* w, tern_half* out, tern_stream stream) {
    const tern_status st = check_nib(w);
    if (st != TERN_OK) return st;
    if (!out) return TERN_ERR_NULL;
    if (!aligned16(out)) return TERN_ERR_ALIGN;
    auto kernel = w->group == 32 ? dequant_kernel<32> : w->group == 64 ? dequant_kernel<64> : dequant_kernel<128>;
    return launch_dependent(kernel, blocks_for(w->N, w->K), kThreads, as_cuda(stream), w->codes, reinterpret_cast<const __half*>(w->scale),
                            reinterpret_cast<const __half*>(w->mu), w->N, w->K, reinterpret_cast<__half*>(out));
}

extern "C" tern_status tern_nib_pack(const uint8_t* c, const tern_half* s, const tern_half* m, int64_t N, int64_t K,
                                     int32_t group, uint32_t* codes, tern_half* scale, tern_half* mu,
                                     tern_stream stream) {
    tern_status st = check_shape(N, K, group);
    if (st != TERN_OK) return st;
    if (!c || !s || !codes || !scale || (m != nullptr) != (mu != nullptr)) return TERN_ERR_NULL;
    if (!aligned16(c) || !aligned16(s) || !aligned16(codes) || !aligned16(scale) || (m && (!aligned16(m) || !aligned16(mu))))
        return TERN_ERR_ALIGN;
    cudaStream_t cs = as_cuda(stream);
    unsigned int* flag = acquire_flag_slot(cs);
    if (!flag) return TERN_ERR_CUDA;
    auto kernel = group == 32 ? pack_kernel<32> : group == 64 ? pack_kernel<64> : pack_kernel<128>;
    kernel<<<blocks_for(N, K), kThreads, 0, cs>>>(c, reinterpret_cast<const __half*>(s), reinterpret_cast<const __half*>(m),
                                                  N, K, codes, reinterpret_cast<__half*>(scale),
                                                  reinterpret_cast<__half*>(mu), flag);
    if ((st = launched()) != TERN_OK) return st;
    unsigned int bad = 0;
    if ((st = read_flag_slot(flag, cs, &bad)) != TERN_OK) return st;
    return bad ? TERN_ERR_BAD_CODE : TERN_OK;
}
