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

// Code of x for step s and zero z: rint((x - z) / s) + bias in 0 .. 15, the quotient rounded to fp32 first;
// inv = 1 / s to fp32. t is within 1e-5 of that quotient for every |t| < 32, so unless it lies next to a
// tie both round to the same integer; the division is done only there.
__device__ __forceinline__ int code_of(float x, float z, float s, float inv, int bias) {
    const float d = __fsub_rn(x, z);
    float t = __fmul_rn(d, inv);
    const float r = rintf(t);
    if (fabsf(fabsf(__fsub_rn(t, r)) - 0.5f) < 1e-4f) t = __fdiv_rn(d, s);
    const float c = fminf(fmaxf(rintf(t) + float(bias), 0.f), 15.f);
    return int(c);
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

inline tern_status launched() { return cudaGetLastError() == cudaSuccess ? TERN_OK : TERN_ERR_CUDA; }

}  // namespace nib
}  // namespace tern
