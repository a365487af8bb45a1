// Pieces shared by the 4-bit operators (weights and cache): codes to fp16 pairs, the fit of one
// group, and host checks.
#pragma once

#include "tern_device.cuh"

namespace tern {
namespace nib {

using namespace dev;

constexpr int kBlockWords = 256;           // words of one (strip, 128 columns) block of a weight

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Pair P (0 .. 3) of a word's codes, nibbles P and P + 4, as fp16 (c - kBias), exactly: a LOP3 puts both
// under the exponent of 1024, where a code in bits 0-3 counts 1 and one in bits 4-7 counts 16, and one
// fp16 operation takes the rest away. w8 = w >> 8. kBias is 8 (weights) or 0 (cache).
template <int P, int kBias>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t w8) {
    const uint32_t v = P < 2 ? w : w8;
    if ((P & 1) == 0) {
        const __half2 h = as_h2(lop3_and_or(v, 0x000F000Fu, 0x64006400u));
        return as_u32(__hsub2(h, as_h2(kBias ? 0x64086408u : 0x64006400u)));                       // 1032 or 1024
    }
    const __half2 h = as_h2(lop3_and_or(v, 0x00F000F0u, 0x64006400u));
    return as_u32(__hfma2(h, as_h2(0x2C002C00u), as_h2(kBias ? 0xD480D480u : 0xD400D400u)));       // / 16 - 72 or - 64
}

// Pair P of a word's codes plus 64, exactly: codes in bits 4-7 under the exponent of 64 count 1 each; those in bits
// 0-3 come under that of 1024 and lose 960. Two operations fewer a word than code_pair; what the 64 add to a product,
// 64 times the other factor's sum, is taken off in fp32 behind the sum.
template <int P>
__device__ __forceinline__ uint32_t code_pair_64(uint32_t w, uint32_t w8) {
    const uint32_t v = P < 2 ? w : w8;
    if (P & 1) return lop3_and_or(v, 0x00F000F0u, 0x54005400u);
    return as_u32(__hsub2(as_h2(lop3_and_or(v, 0x000F000Fu, 0x64006400u)), as_h2(0x63806380u)));
}

// D += A . B for one m16n8k16 tile, fp16 inputs, fp32 accumulators. Not volatile: the compiler may move it among the
// loads and decodes of other steps.
__device__ __forceinline__ void mma_next(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A . B: the first step of a sum, with nothing to clear.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// D += A . B for one m16n8k8 tile of tf32 values held in fp32: fp16 numbers are exact in it. Lane 4 g + q holds
// A (rows g and g + 8, column q), (.., column q + 4) and B (row q, column g), (row q + 4, column g).
__device__ __forceinline__ void mma_1688(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

__device__ __forceinline__ void mma_1688_first(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)), "f"(0.f));
}

// v = hi + lo, each a tf32 number, but for 2^-22 v.
__device__ __forceinline__ float tf32_part(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFFE000u); }

// ---------------------------------------------------------------- quantising
// Codes of eight neighbouring fp16 values for step s and zero z: rint((x - z) / s) + kBias in 0 .. 15, the quotient rounded
// to fp32 first, column i at nibble i / 2 + 4 (i % 2) (kPlain: at nibble i). inv = 1 / s to an ulp. With no bias x >= z is
// the caller's.
//
// The quotient is q + r inv with q = (x - z) inv and the exact remainder r = (x - z) - q s, rounded once: that is off the
// true one by less than 2^-21 ulp, and a quotient by the 11 bits of a step is at least 2^-12 ulp from every midpoint of two
// fp32 numbers, so it is the IEEE quotient. It is rounded by adding 1.5 2^23 (to nearest, ties to even), whose bits then carry
// the code.
template <int kBias, bool kPlain = false>
__device__ __forceinline__ uint32_t codes_of(uint4 v, float z, float s, float inv) {
    constexpr float kMagic = 12582912.f + float(kBias);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t w = 0, upper = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(as_h2(u[i / 2]));
        const float d = __fsub_rn(i & 1 ? f.y : f.x, z), q = __fmul_rn(d, inv);
        const float m = __fadd_rn(__fmaf_rn(__fmaf_rn(-q, s, d), inv, q), kMagic);
        int c = min(__float_as_int(m), 0x4B40000F);                 // the code in the low bits
        if (kBias) c = max(c, 0x4B400000);
        const int at = 4 * (kPlain ? i : i / 2 + 4 * (i & 1));
        w += uint32_t(c) << at;
        upper += 0x4B400000u << at;        // the upper bits, shifted as the codes are (modulo 2^32)
    }
    return w - upper;
}

// 1 / s to an ulp.
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}

// x / kBy as the IEEE division rounds it: a quotient by the reciprocal, and the exact remainder's share. (Checked over every
// fp32 mantissa for 15 and 7; x is 0 or at least 2^-24, or not finite: then so is the result.)
template <int kBy>
__device__ __forceinline__ float divided(float x) {
    constexpr float r = 1.f / float(kBy);
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, float(kBy), x), r, q);
}

// Smallest and largest of values seen so far; a NaN stays.
__device__ __forceinline__ void take_range(uint4 v, __half2& lo, __half2& hi) {
    lo = __hmin2_nan(lo, __hmin2_nan(__hmin2_nan(as_h2(v.x), as_h2(v.y)), __hmin2_nan(as_h2(v.z), as_h2(v.w))));
    hi = __hmax2_nan(hi, __hmax2_nan(__hmax2_nan(as_h2(v.x), as_h2(v.y)), __hmax2_nan(as_h2(v.z), as_h2(v.w))));
}

// Over the pair and the `lanes` lanes that share it (a power of two): (lo, hi) of all.
template <int kLanes>
__device__ __forceinline__ float2 whole_range(__half2 lo, __half2 hi) {
    __half2 r = __halves2half2(__hmin_nan(__low2half(lo), __high2half(lo)), __hneg(__hmax_nan(__low2half(hi), __high2half(hi))));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) r = __hmin2_nan(r, as_h2(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    return make_float2(__low2float(r), -__high2float(r));
}

inline bool overlaps(const void* a, size_t abytes, const void* b, size_t bbytes) {
    const uintptr_t ab = reinterpret_cast<uintptr_t>(a), bb = reinterpret_cast<uintptr_t>(b);
    return ab < bb + bbytes && bb < ab + abytes;
}

constexpr int64_t kMaxRows = int64_t(1) << 22;     // the ternary weights' limits
constexpr int64_t kMaxK = int64_t(1) << 20;

inline tern_status check_shape(int64_t N, int64_t K, int32_t group) {
    if (N <= 0 || K <= 0 || K % kGroup || N > kMaxRows || K > kMaxK) return TERN_ERR_SHAPE;
    return group == 32 || group == 64 || group == 128 ? TERN_OK : TERN_ERR_SHAPE;
}

inline tern_status check_nib(const tern_nib_weight* w) {
    if (!w) return TERN_ERR_NULL;
    const tern_status s = check_shape(w->N, w->K, w->group);
    if (s != TERN_OK) return s;
    if (!w->codes || !w->scale) return TERN_ERR_NULL;
    if (!aligned16(w->codes) || !aligned16(w->scale) || (w->mu && !aligned16(w->mu))) return TERN_ERR_ALIGN;
    return TERN_OK;
}

// Launches a kernel that waits for the one before it itself (programmatic dependent launch).
template <typename... P, typename... A>
inline tern_status launch_dependent(void (*kernel)(P...), unsigned ctas, unsigned threads, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? TERN_OK : TERN_ERR_CUDA;
}

inline tern_status launched() { return cudaGetLastError() == cudaSuccess ? TERN_OK : TERN_ERR_CUDA; }

}  // namespace nib
}  // namespace tern
