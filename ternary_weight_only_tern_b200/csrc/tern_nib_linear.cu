// y [M, N] = x [M, K] . W^T for a 4-bit W = mu + s (c - 8) and up to 16 tokens (tern.h has the layout; more tokens go to
// tern_nib_gemm.cu).
//
//   y[m, n] = sum_g s[n, g] sum_{k in g} (c[n, k] - 8) x[m, k] + mu[n, g] sum_{k in g} x[m, k].
// The inner sums run on mma.sync m16n8k16 with a strip's 16 rows of codes plus 64, exact in fp16, as A and 8 tokens as
// B's columns; a group's accumulators are scaled in fp32. The 72 too much and the offset, -72 s X + mu X with X = sum x
// of the group, are four fp32 operations per group and token pair, and at group 32 a product of their own: two m16n8k8
// in tf32 per block of 128 columns, where s and mu are exact and X is taken in two parts (65543 x 2560, 6 tokens: 24.9 us
// against 27.6; at group 64 the plain form: 131072 x 4096, 16 tokens, 91.7 against 119.4). The layout
// is that of A: one 16-byte shared-memory read gives a lane its four words, a word is four pairs of neighbouring
// columns, and x is read as it lies.
//
// Bound by HBM (N K / 2 bytes and the scales), next by the issue of the decoding. A resident grid walks the strips; in a
// CTA a producer warp runs ahead with bulk copies of up to 32 of a strip's blocks of 128 columns, which are contiguous, into
// a ring of stages (copies of 2 KB and less, one set per warp, were bound by their number: about 73 cycles each on an
// SM), eight warps take the blocks in turn, counted on over the strips so that their shares even out for any K, and an
// epilogue warp adds the eight warps' sums of a strip, in warp order, and writes y while they go on. x stays in
// shared memory, rows 64 bytes apart modulo 128, so that a fragment's reads hit all banks once. Where x is too large for
// that the columns are cut into slices, a grid row each, whose sums go to the workspace in fp32 and are added by a
// second kernel. With static weights the ring fills before the wait on the previous kernel.
// Measured: 131072 x 4096, group 128, 1 token 53.9 us (5.1 TB/s), 8 tokens 60.6; 12288 x 4096 9.0 us; 65543 x 2560, group 32
// with offsets, 6 tokens 24.8 us (4.3 TB/s). Sixteen warps in one CTA, or in groups that share a strip, were slower.
#include <algorithm>
#include <mutex>

#include "tern_nib.cuh"
#include "tern_stream.cuh"

namespace tern {
namespace nib {

// tern_nib_gemm.cu
tern_status gemm_launch(const tern_nib_weight& w, const __half* x, int64_t M, __half* y, void* workspace, cudaStream_t stream);
void add_slices(const float* part, int slices, int64_t n, __half* y, cudaStream_t stream, cudaError_t& err);
size_t gemm_workspace_bytes(const tern_nib_weight& w, int64_t M);

}  // namespace nib

namespace {

using namespace nib;

constexpr int kWarps = 8;                  // that multiply
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kMaxStages = 4;
constexpr int kStageBlocks = 32;           // blocks of 128 columns in a stage at most
constexpr int64_t kMaxM = 16;
constexpr int64_t kMostTokens = int64_t(1) << 22;    // of a call: 65535 tiles of the least rows many tokens get, 128, hold them
constexpr int kTf32Per = 4;                // groups of a block from which the correction is a tf32 product

struct Args {
    const uint32_t* codes;
    const __half* scale;
    const __half* mu;
    const __half* x;
    __half* y;
    float* part;               // [gridDim.y][M][N] sums of a slice of the columns, or nullptr (gridDim.y == 1)
    int64_t N;
    int M;
    int KB, strips;            // blocks of 128 columns, strips of 16 rows
    int slice;                 // blocks per slice
    int stage_blocks, stages, stage_bytes;
    int x_off, sum_off, ring_off, red_off;     // shared memory, bytes
    int early;                 // the weights may be read before the previous kernel has ended
    unsigned int* status;
};

__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bulk(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                 "l"(reinterpret_cast<uint64_t>(from)), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int kGrp, int NT>
__global__ void __launch_bounds__(kThreads, 2) linear_kernel(const Args a) {
    constexpr int per = kGroup / kGrp, span = kGrp / 32, kPitch = 8 * NT + 1, kRed = 16 * kPitch;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);            // full and empty of the stages and of the two sums, x's
    const uint32_t at = smem_u32(smem);
    const uint32_t full = at, empty = full + kMaxStages * 8, red_full = empty + kMaxStages * 8, red_empty = red_full + 16,
                   x_bar = red_empty + 16;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(bars + i, 1);
            mbar_init(bars + kMaxStages + i, kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + 2 * kMaxStages + i, kWarps);
            mbar_init(bars + 2 * kMaxStages + 2 + i, 1);
        }
        mbar_init(bars + 2 * kMaxStages + 4, 1);
        fence_barrier_init();
    }
    __syncthreads();
    grid_launch_dependents();

    const int kb0 = int(blockIdx.y) * a.slice, nb = min(a.slice, a.KB - kb0), M = a.M;
    const int per_strip = (nb + a.stage_blocks - 1) / a.stage_blocks;      // stages of a strip
    const int rounds = (a.strips - int(blockIdx.x) + int(gridDim.x) - 1) / int(gridDim.x);
    const int pitch = a.slice * kGroup * 2 + 64;
    const int scale_off = a.stage_blocks * kBlockWords * 4, mu_off = scale_off + a.stage_blocks * per * 32;
    bool ok = true;

    if (warp == kWarps) {
        // ---- producer
        int stage = 0, round = 0, s = 0;
        uint32_t phase = 1;
        const int items = rounds * per_strip;
        auto issue = [&](int i) {
            if (i >= a.stages) ok = ok && stream::mbar_poll_addr(empty + stage * 8, phase, 64);
            const int n = min(a.stage_blocks, nb - s * a.stage_blocks);
            const int64_t blk = int64_t(int(blockIdx.x) + round * int(gridDim.x)) * a.KB + kb0 + s * a.stage_blocks;
            const uint32_t bar = full + stage * 8, to = at + a.ring_off + stage * a.stage_bytes;
            if (lane == 0 && ok) {
                expect(bar, uint32_t(n) * (kBlockWords * 4 + (a.mu ? 2 : 1) * per * 32));
                bulk(to, a.codes + blk * kBlockWords, n * kBlockWords * 4, bar);
                bulk(to + scale_off, a.scale + blk * per * 16, n * per * 32, bar);
                if (a.mu) bulk(to + mu_off, a.mu + blk * per * 16, n * per * 32, bar);
            }
            if (++s == per_strip) s = 0, ++round;
            if (++stage == a.stages) stage = 0, phase ^= 1u;
        };
        int i = 0;
        if (a.early)
            for (; i < items && i < a.stages; ++i) issue(i);
        grid_dependency_wait();
        if (lane == 0) expect(x_bar, uint32_t(M * nb * kGroup * 2));
        __syncwarp();
        if (lane < M) bulk(at + a.x_off + lane * pitch, a.x + (int64_t(lane) * a.KB + kb0) * kGroup, nb * kGroup * 2, x_bar);
        for (; i < items && ok; ++i) issue(i);
        if (!ok)       // a wait ran out: the copies under way land before the CTA ends
            for (int j = max(0, i - 1 - a.stages); j < i - 1; ++j) stream::mbar_poll_addr(full + j % a.stages * 8, j / a.stages & 1, 0);
    } else if (warp < kWarps) {
        // ---- the products
        const int g = lane >> 2, q = lane & 3;
        ok = mbar_wait(bars + 2 * kMaxStages + 4, 0);
        float4* sums = reinterpret_cast<float4*>(smem + a.sum_off);        // [nb per][8 NT] -72 X and X of a group, in two parts
        float2* plain = reinterpret_cast<float2*>(smem + a.sum_off);       // or X alone, [nb per][8 NT / 2]
        // the lane's token of each 8 (a token past the last repeats it: its columns are never written)
        const uint8_t* xa[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xa[t] = smem + a.x_off + min(8 * t + g, M - 1) * pitch + q * 16;
        for (int kb = warp; kb < nb; kb += kWarps) {
            const uint32_t one[4] = {kHalf2One, kHalf2One, kHalf2One, kHalf2One};
#pragma unroll
            for (int j0 = 0; j0 < 4; j0 += span)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = j0; j < j0 + span; ++j) {
                        const uint4 xv = *reinterpret_cast<const uint4*>(xa[t] + kb * (kGroup * 2) + j * 64);
                        mma_next(acc, one, xv.x, xv.y);
                        mma_next(acc, one, xv.z, xv.w);
                    }
                    if (g == 0) {
                        if constexpr (per != kTf32Per) {
                            plain[(kb * per + j0 / span) * 8 * NT / 2 + 4 * t + q] = make_float2(acc[0], acc[1]);
                        } else {
                            float4* to = sums + (kb * per + j0 / span) * 8 * NT + 8 * t + 2 * q;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float X = acc[i], Y = -72.f * X, xh = tf32_part(X), yh = tf32_part(Y);
                                to[i] = make_float4(yh, xh, tf32_part(Y - yh), tf32_part(X - xh));
                            }
                        }
                    }
                }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        int stage = 0, first = warp;       // first: of this warp's blocks in the strip
        uint32_t phase = 0;
        for (int round = 0; round < rounds; ++round) {
            float sum[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[t][0] = sum[t][1] = sum[t][2] = sum[t][3] = 0.f;
            int kb = first;                // within the slice
            for (int s = 0; s < per_strip; ++s) {
                ok = ok && stream::mbar_poll_addr(full + stage * 8, phase, 0);
                const uint8_t* ring = smem + a.ring_off + stage * a.stage_bytes;
                const int b0 = s * a.stage_blocks, b1 = min(nb, b0 + a.stage_blocks);
                for (; kb < b1; kb += kWarps) {
                    const int b = kb - b0;
                    const uint4* from = reinterpret_cast<const uint4*>(ring + b * (kBlockWords * 4)) + lane;
                    const uint4 u = from[0], v = from[32];
                    const uint32_t wa[4] = {u.x, u.y, u.z, u.w}, wb[4] = {v.x, v.y, v.z, v.w};
                    const __half2* sc_at = reinterpret_cast<const __half2*>(ring + scale_off + b * per * 32) + g;
                    if constexpr (per == kTf32Per) {
                        // column q of the tf32 product: group q of the block (none from `per` on)
                        float2 sq = make_float2(0.f, 0.f), mq = make_float2(0.f, 0.f);
                        if (q < per) {
                            sq = __half22float2(sc_at[q * 8]);
                            if (a.mu) mq = __half22float2(sc_at[(mu_off - scale_off) / 4 + q * 8]);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float4 xs = sums[(kb * per + (q < per ? q : 0)) * 8 * NT + 8 * t + g];
                            mma_1688(sum[t], sq.x, sq.y, mq.x, mq.y, xs.x, xs.y);
                            mma_1688(sum[t], sq.x, sq.y, mq.x, mq.y, xs.z, xs.w);
                        }
                    }
#pragma unroll
                    for (int j0 = 0; j0 < 4; j0 += span) {
                        float acc[NT][4];
#pragma unroll
                        for (int j = j0; j < j0 + span; ++j) {
                            const uint32_t a8 = wa[j] >> 8, b8 = wb[j] >> 8;
                            const uint32_t A0[4] = {code_pair_64<0>(wa[j], a8), code_pair_64<0>(wb[j], b8),
                                                    code_pair_64<1>(wa[j], a8), code_pair_64<1>(wb[j], b8)};
                            const uint32_t A1[4] = {code_pair_64<2>(wa[j], a8), code_pair_64<2>(wb[j], b8),
                                                    code_pair_64<3>(wa[j], a8), code_pair_64<3>(wb[j], b8)};
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const uint4 xv = *reinterpret_cast<const uint4*>(xa[t] + kb * (kGroup * 2) + j * 64);
                                if (j == j0) mma_first(acc[t], A0, xv.x, xv.y);
                                else mma_next(acc[t], A0, xv.x, xv.y);
                                mma_next(acc[t], A1, xv.z, xv.w);
                            }
                        }
                        const float2 sc = __half22float2(sc_at[j0 / span * 8]);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            sum[t][0] += sc.x * acc[t][0];
                            sum[t][1] += sc.x * acc[t][1];
                            sum[t][2] += sc.y * acc[t][2];
                            sum[t][3] += sc.y * acc[t][3];
                        }
                        if constexpr (per != kTf32Per) {
                            float2 mu = make_float2(-72.f * sc.x, -72.f * sc.y);
                            if (a.mu) {
                                const float2 f = __half22float2(sc_at[(mu_off - scale_off) / 4 + j0 / span * 8]);
                                mu.x += f.x;
                                mu.y += f.y;
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const float2 X = plain[(kb * per + j0 / span) * 8 * NT / 2 + 4 * t + q];
                                sum[t][0] += mu.x * X.x;
                                sum[t][1] += mu.x * X.y;
                                sum[t][2] += mu.y * X.x;
                                sum[t][3] += mu.y * X.y;
                            }
                        }
                    }
                }
                __syncwarp();       // every lane has read the stage
                if (lane == 0) stream::mbar_arrive_addr(empty + stage * 8);
                if (++stage == a.stages) stage = 0, phase ^= 1u;
            }
            first = kb - nb;        // the next block in turn, in the next strip
            // ---- hand the strip's sums over
            const int buf = round & 1;
            if (round >= 2) ok = ok && stream::mbar_poll_addr(red_empty + buf * 8, ((round >> 1) - 1) & 1, 0);
            float* mine = reinterpret_cast<float*>(smem + a.red_off) + (buf * kWarps + warp) * kRed;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 8 * t + 2 * q + (i & 1);
                    if (m < M) mine[(g + 8 * (i >> 1)) * kPitch + m] = sum[t][i];
                }
            __syncwarp();
            if (lane == 0) stream::mbar_arrive_addr(red_full + buf * 8);
        }
    } else {
        // ---- epilogue: row lane % 16, tokens lane / 16, + 2, ..
        for (int round = 0; round < rounds; ++round) {
            const int buf = round & 1, row = lane & 15;
            ok = ok && stream::mbar_poll_addr(red_full + buf * 8, (round >> 1) & 1, 64);
            const float* all = reinterpret_cast<const float*>(smem + a.red_off) + buf * kWarps * kRed + row * kPitch;
            const int64_t n = (int64_t(blockIdx.x) + int64_t(round) * gridDim.x) * 16 + row;
            for (int m = lane >> 4; m < M; m += 2) {
                float f = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) f += all[w * kRed + m];
                if (n < a.N) {
                    if (a.part) a.part[(int64_t(blockIdx.y) * M + m) * a.N + n] = f;
                    else a.y[int64_t(m) * a.N + n] = __float2half_rn(f);
                }
            }
            __syncwarp();
            if (lane == 0) stream::mbar_arrive_addr(red_empty + buf * 8);
        }
    }
    if (!ok && a.status) atomicOr(a.status, kStatusTimeout);
}

// y = the sum of the slices' parts, in order.
__global__ void __launch_bounds__(256) add_kernel(const float* __restrict__ part, int slices, int64_t n, __half* __restrict__ y) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    float f = 0.f;
    for (int s = 0; s < slices; ++s) f += part[s * n + i];
    y[i] = __float2half_rn(f);
}

}  // namespace

namespace nib {

void add_slices(const float* part, int slices, int64_t n, __half* y, cudaStream_t stream, cudaError_t& err) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((n + 255) / 256), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, add_kernel, part, slices, n, y);
}

}  // namespace nib

namespace {

// ---------------------------------------------------------------- the plan of a call
constexpr int kSmemMax = 227 * 1024;

struct Plan {
    int nt, slices, slice, stage_blocks, stages, stage_bytes, x_off, sum_off, ring_off, red_off, smem, per_sm;
};

// Shared memory of a plan with the given slices and stages; false where it is too much.
bool layout(const tern_nib_weight& w, int M, Plan& p, int slices, int stages, int stage_blocks, int64_t limit) {
    const int KB = int(w.K / kGroup), per = kGroup / w.group;
    p.slice = (KB + slices - 1) / slices;
    p.slices = (KB + p.slice - 1) / p.slice;
    const int per_strip = (p.slice + stage_blocks - 1) / stage_blocks;
    p.stage_blocks = (p.slice + per_strip - 1) / per_strip;
    p.stages = stages;
    auto up = [](int64_t b) { return (b + 127) & ~int64_t(127); };
    p.stage_bytes = int(up(int64_t(p.stage_blocks) * (kBlockWords * 4 + (w.mu ? 2 : 1) * per * 32)));
    int64_t at = 128;
    p.x_off = int(at);
    at = up(at + int64_t(M) * (int64_t(p.slice) * kGroup * 2 + 64));
    if (at > limit) return false;
    p.sum_off = int(at);
    at = up(at + int64_t(p.slice) * per * 8 * p.nt * (per == kTf32Per ? 16 : 4));
    p.ring_off = int(at);
    at = up(at + int64_t(stages) * p.stage_bytes);
    p.red_off = int(at);
    at = up(at + int64_t(2) * kWarps * 16 * (8 * p.nt + 1) * 4);
    if (at > limit) return false;
    p.smem = int(at);
    return true;
}

// As few slices as x allows; two CTAs per SM where the rings of both fit beside x, else one; large stages before many
// (M = 1, K = 4096, 131072 rows: two stages of 32 blocks 58 us, four of 16 62 us).
bool plan_of(const tern_nib_weight& w, int M, Plan& p) {
    p.nt = M <= 8 ? 1 : 2;
    for (int slices = 1; slices <= int(w.K / kGroup); ++slices)
        for (p.per_sm = 2; p.per_sm >= 1; --p.per_sm)
            for (int blocks = kStageBlocks; blocks >= 8; blocks -= 8)
                for (int stages = kMaxStages; stages >= 2; --stages)
                    if (layout(w, M, p, slices, stages, blocks, kSmemMax / p.per_sm)) return true;
    return false;
}

template <int kGrp, int NT>
tern_status launch(const Plan& p, Args& a, cudaStream_t stream) {
    static std::mutex mu;
    static bool configured[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TERN_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev]) {
            if (cudaFuncSetAttribute(linear_kernel<kGrp, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
                return TERN_ERR_CUDA;
            configured[dev] = true;
        }
    }
    const int fill = std::max(1, sm_count() * p.per_sm / p.slices);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min(a.strips, fill)), unsigned(p.slices), 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = size_t(p.smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, linear_kernel<kGrp, NT>, a) != cudaSuccess) return TERN_ERR_CUDA;
    if (p.slices == 1) return TERN_OK;
    cudaError_t err;
    add_slices(a.part, p.slices, int64_t(a.M) * a.N, a.y, stream, err);
    return err == cudaSuccess ? TERN_OK : TERN_ERR_CUDA;
}

}  // namespace
}  // namespace tern

using namespace tern;
using namespace tern::nib;

extern "C" size_t tern_nib_linear_workspace_bytes(const tern_nib_weight* w, int64_t M) {
    if (check_nib(w) != TERN_OK || M <= 0) return 0;
    if (M > kMaxM) return gemm_workspace_bytes(*w, M);
    Plan p;
    if (!plan_of(*w, int(M), p) || p.slices == 1) return 0;
    return (size_t(p.slices) * size_t(M) * size_t(w->N) * 4 + 255) & ~size_t(255);
}

extern "C" tern_status tern_nib_linear(const tern_nib_weight* w, const tern_half* x, int64_t M, tern_half* y,
                                       void* workspace, size_t workspace_bytes, tern_stream stream) {
    const tern_status st = check_nib(w);
    if (st != TERN_OK) return st;
    if (M < 0 || M > kMostTokens) return TERN_ERR_SHAPE;
    if (M == 0) return TERN_OK;
    if (!x || !y) return TERN_ERR_NULL;
    if (!aligned16(x) || !aligned16(y)) return TERN_ERR_ALIGN;
    const size_t need = tern_nib_linear_workspace_bytes(w, M);
    if (need && (!workspace || workspace_bytes < need)) return TERN_ERR_WORKSPACE;
    if (workspace && !aligned16(workspace)) return TERN_ERR_ALIGN;
    if (overlaps(x, size_t(M) * size_t(w->K) * 2, y, size_t(M) * size_t(w->N) * 2)) return TERN_ERR_SHAPE;
    const __half* xh = reinterpret_cast<const __half*>(x);
    __half* yh = reinterpret_cast<__half*>(y);
    cudaStream_t cs = as_cuda(stream);
    if (M > kMaxM) return gemm_launch(*w, xh, M, yh, workspace, cs);
    Plan p;
    if (!plan_of(*w, int(M), p)) return TERN_ERR_SHAPE;
    Args a{};
    a.codes = w->codes;
    a.scale = reinterpret_cast<const __half*>(w->scale);
    a.mu = reinterpret_cast<const __half*>(w->mu);
    a.x = xh;
    a.y = yh;
    a.part = p.slices > 1 ? static_cast<float*>(workspace) : nullptr;
    a.N = w->N;
    a.M = int(M);
    a.KB = int(w->K / kGroup);
    a.strips = int((w->N + 15) / 16);
    a.slice = p.slice;
    a.stage_blocks = p.stage_blocks;
    a.stages = p.stages;
    a.stage_bytes = p.stage_bytes;
    a.x_off = p.x_off;
    a.sum_off = p.sum_off;
    a.ring_off = p.ring_off;
    a.red_off = p.red_off;
    a.early = (w->flags & TERN_WEIGHT_STATIC) != 0;
    a.status = async_status_word();
    if (p.nt == 1) return w->group == 32 ? launch<32, 1>(p, a, cs) : w->group == 64 ? launch<64, 1>(p, a, cs) : launch<128, 1>(p, a, cs);
    return w->group == 32 ? launch<32, 2>(p, a, cs) : w->group == 64 ? launch<64, 2>(p, a, cs) : launch<128, 2>(p, a, cs);
}
