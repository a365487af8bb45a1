// y [M, N] = x [M, K] . W^T for a 4-bit W = mu + s (c - 8) (tern.h has the layout).
//
// One warp takes a strip of 16 rows and 8 tokens: mma.sync m16n8k16 with the strip's codes as A (exact in fp16)
// and the tokens as B's columns, fp32 accumulators per group, then
//   y[m, n] = sum_g s[n, g] sum_k (c - 8) x + mu[n, g] sum_k x,
// the second sum from the same instruction with A = 1.
#include "tern_nib.cuh"

namespace tern {
namespace {

using namespace nib;

constexpr int kWarps = 4;

template <int kGrp>
__global__ void __launch_bounds__(kWarps * 32) linear_kernel(const uint32_t* __restrict__ codes,
                                                             const __half* __restrict__ scale,
                                                             const __half* __restrict__ mu, int64_t N, int64_t K,
                                                             const __half* __restrict__ x, int64_t M,
                                                             __half* __restrict__ y) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int64_t strip = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5), KB = K / kGroup;
    const int64_t m0 = int64_t(blockIdx.y) * 8;
    if (strip * 16 >= N) return;
    const bool token = m0 + g < M;
    const __half* xr = x + (token ? m0 + g : 0) * K + 8 * q;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int span = kGrp / 32;
    for (int64_t kb = 0; kb < KB; ++kb) {
        const uint32_t* block = codes + (strip * KB + kb) * kBlockWords + lane * 4;
        const uint4 va = __ldg(reinterpret_cast<const uint4*>(block));
        const uint4 vb = __ldg(reinterpret_cast<const uint4*>(block + 128));
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += span) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f}, ones[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = j0; j < j0 + span; ++j) {
                const uint4 b = token ? __ldg(reinterpret_cast<const uint4*>(xr + kb * kGroup + 32 * j))
                                      : make_uint4(0, 0, 0, 0);
                const uint32_t a8 = wa[j] >> 8, b8 = wb[j] >> 8;
                const uint32_t A0[4] = {code_pair<0, 8>(wa[j], a8), code_pair<0, 8>(wb[j], b8),
                                        code_pair<1, 8>(wa[j], a8), code_pair<1, 8>(wb[j], b8)};
                const uint32_t A1[4] = {code_pair<2, 8>(wa[j], a8), code_pair<2, 8>(wb[j], b8),
                                        code_pair<3, 8>(wa[j], a8), code_pair<3, 8>(wb[j], b8)};
                const uint32_t one[4] = {kHalf2One, kHalf2One, kHalf2One, kHalf2One};
                mma_16816(acc, A0, b.x, b.y);
                mma_16816(acc, A1, b.z, b.w);
                if (mu) {
                    mma_16816(ones, one, b.x, b.y);
                    mma_16816(ones, one, b.z, b.w);
                }
            }
            const int64_t at = ((strip * KB + kb) * (kGroup / kGrp) + j0 / span) * 16 + 2 * g;
            const float2 s = __half22float2(__ldg(reinterpret_cast<const __half2*>(scale + at)));
            sum[0] += s.x * acc[0];
            sum[1] += s.x * acc[1];
            sum[2] += s.y * acc[2];
            sum[3] += s.y * acc[3];
            if (mu) {
                const float2 m = __half22float2(__ldg(reinterpret_cast<const __half2*>(mu + at)));
                sum[0] += m.x * ones[0];
                sum[1] += m.x * ones[1];
                sum[2] += m.y * ones[2];
                sum[3] += m.y * ones[3];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = strip * 16 + g + 8 * (i >> 1), m = m0 + 2 * q + (i & 1);
        if (n < N && m < M) y[m * N + n] = __float2half_rn(sum[i]);
    }
}

}  // namespace

namespace nib {

tern_status gemm_launch(const tern_nib_weight& w, const __half* x, int64_t M, __half* y, cudaStream_t stream) {
    if ((M + 7) / 8 > 65535) return TERN_ERR_SHAPE;
    const dim3 grid(unsigned(((w.N + 15) / 16 + kWarps - 1) / kWarps), unsigned((M + 7) / 8), 1);
    auto kernel = w.group == 32 ? linear_kernel<32> : w.group == 64 ? linear_kernel<64> : linear_kernel<128>;
    kernel<<<grid, kWarps * 32, 0, stream>>>(w.codes, reinterpret_cast<const __half*>(w.scale),
                                             reinterpret_cast<const __half*>(w.mu), w.N, w.K, x, M, y);
    return launched();
}

}  // namespace nib
}  // namespace tern

