// y [M, N] = x [M, K] . W^T for a 4-bit W = mu + s (c - 8) and more than 16 tokens, on tcgen05 tensor cores, W
// dequantised from its codes straight into shared memory (tern.h has the layout).
//
// A CTA computes 128 H weight rows x BT tokens: H tcgen05.mma (kind::f16, M = 128, N = BT, K = 16) per 16 columns of K
// with the weights as A and the tokens as B, fp32 accumulators in H 256 columns of TMEM. Weights as rows: the few
// tokens of a small batch cost few columns, and the layout's 16-byte vectors (32 codes of a row) fit the rows.
// K goes by stages of 128 columns (H = 1) or 64 (H = 2).
//  * warp 0, one thread: TMA loads of the x tile (BT x 64 fp16, 128-byte swizzle) into the stages;
//  * warp 1: issues the MMAs and commits each stage back;
//  * warps 2-17: decode, 16 or 32 rows of a stage each, in groups that take the stages in turn. A lane loads its vectors and
//    scales of its next stage while it works on this one: eight codes are five integer and four fp16 operations,
//    w = rn16(mu + s (c - 8)) four more, and leave as one 16-byte store. Rows of odd index store the other half's word first,
//    so that a quarter warp's stores hit all banks once. The same warps bring the accumulators out of TMEM.
// With few tokens a stage costs its hand-overs (waits, proxy fence, arrivals) more than its MMAs or decoding, hence the
// wide stages and two strips per warp.
// Tile and slices of K are chosen per call by a cost of both sides (plan_of): waves of CTAs times the slower of the MMAs and the
// decoding. The slices' sums go to the workspace in fp32 and are added in order by a second kernel.
// Measured: 2048 tokens, 12288 x 4096, 155 us (1330 TFLOP/s; 181 us in seconds-long runs, under the power cap), the tensor pipe
// active 82 % of the time; 64 tokens 18 us. 384 tiles on 148 SMs are 2.6 waves in the time of 3.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tern_nib.cuh"

namespace tern {
namespace nib {

void add_slices(const float* part, int slices, int64_t n, __half* y, cudaStream_t stream, cudaError_t& err);   // tern_nib_linear.cu

}  // namespace nib

namespace {

using namespace nib;

constexpr int kDecodeWarps = 16;
constexpr int kThreads = (2 + kDecodeWarps) * 32;
constexpr int kMaxStages = 6;
constexpr int kRowsM = 128;                // rows of an MMA
constexpr int kBK = 64;                    // columns of a swizzled tile
constexpr int kABytes = kRowsM * kBK * 2;
constexpr int kBKs(int H) { return H == 1 ? 2 : 1; }               // tiles of a stage
constexpr int kSmemMax = 227 * 1024;

struct Args {
    const uint32_t* codes;
    const __half* scale;
    const __half* mu;
    __half* y;
    float* part;               // [gridDim.z][M][N], or nullptr
    int64_t N, M;
    int KB, strips, slice;     // blocks of 128 columns; of a slice
    int bt, stages, stage_bytes;
    int early;
    unsigned int* status;
};

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr) {
    return ((uint64_t(addr) & 0x3FFFFull) >> 4) | (1ull << 16) | (uint64_t(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// One MMA, issued by one lane of a converged warp: the operands are then uniform registers as they stand (issued from a
// single-lane branch each took about 90 cycles to gather them).
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void load_tmem32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// kStrips: strips that a decoding warp takes of a stage. The groups of warps that take the stages in turn, kSets, are at most
// as many as the stages: a group's wait for a stage then follows one that says the stage's last use but one is over, so
// that a barrier's parity is never a whole turn behind.
template <int kGrp, int H, int kStrips>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const Args a) {
    constexpr int per = kGroup / kGrp, kTiles = kBKs(H);  // groups of a block; tiles of a stage
    constexpr int kSets = kDecodeWarps * kStrips / (8 * H);  // groups of decoding warps (the caller: stages >= kSets)
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
    __shared__ uint32_t tmem_slot;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n0 = int64_t(blockIdx.x) * kRowsM * H, m0 = int64_t(blockIdx.y) * a.bt;
    const int kb0 = int(blockIdx.z) * a.slice, nb = min(a.slice, a.KB - kb0), steps = nb * 2 / kTiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&full[s], 8 * H / kStrips + 1);     // the decoding warps and x's loader
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(256 * H) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot, base = smem_u32(smem);
    grid_launch_dependents();
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            grid_dependency_wait();
            int issued = 0;
            for (int i = 0, s = 0, ph = 1; i < steps; ++i) {
                if (i >= a.stages) ok = mbar_wait(&empty[s], ph);
                if (!ok) break;
                mbar_arrive_expect_tx(&full[s], uint32_t(kTiles * a.bt * kBK * 2));
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
                    tma_load_2d(smem + s * a.stage_bytes + kTiles * H * kABytes + j * a.bt * kBK * 2, &tmap_x, (kb0 * 2 + i * kTiles + j) * kBK,
                                int(m0), &full[s]);
                issued = i + 1;
                if (++s == a.stages) s = 0, ph ^= 1;
            }
            // every copy lands before the CTA may end
            for (int i = max(0, issued - a.stages); i < issued; ++i) ok = mbar_wait_for(&full[i % a.stages], (i / a.stages) & 1, ok ? kWaitLimitCycles : kWaitLimitCycles / 64) && ok;
        }
    } else if (warp == 1) {
        const uint32_t idesc = (1u << 4) | (uint32_t(a.bt >> 3) << 17) | (uint32_t(kRowsM >> 4) << 24);
        const uint32_t d = __shfl_sync(0xffffffffu, tmem, 0), at0 = __shfl_sync(0xffffffffu, base, 0);
        const uint32_t empty_at = __shfl_sync(0xffffffffu, smem_u32(empty), 0);
        for (int i = 0, s = 0, ph = 0; i < steps; ++i) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ph));
            if (!ok) break;
            fence_after();
            const uint32_t at = at0 + s * a.stage_bytes;
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                const uint64_t wd = matrix_desc(at + j * H * kABytes), xd = matrix_desc(at + kTiles * H * kABytes + j * a.bt * kBK * 2);   // + 2: 32 bytes on
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
#pragma unroll
                    for (int h = 0; h < H; ++h) mma_f16(d + 256 * h, wd + (h * kABytes >> 4) + 2 * k, xd + 2 * k, idesc, i > 0 || j > 0 || k > 0);
            }
            commit(empty_at + s * 8);
            if (++s == a.stages) s = 0, ph ^= 1;
        }
        commit(smem_u32(&done));          // also after a timeout: every issued MMA retires first
        if (!mbar_wait(&done, 0)) ok = false;
    } else {
        // ---- decode: kStrips strips of every kSets-th stage; vector 2 h + v: strip h, rows 8 v + g
        constexpr int kWords = 2 * kTiles, kGrps = kWords * 32 > kGrp ? kWords * 32 / kGrp : 1;   // a vector's words and groups in a stage
        const int dw = (warp - 2) % (8 * H / kStrips), set = (warp - 2) / (8 * H / kStrips), g = lane >> 2, q = lane & 3;
        const uint32_t* from[kStrips];
        const __half2* sc[kStrips];
        const __half2* mu[kStrips];
#pragma unroll
        for (int h = 0; h < kStrips; ++h) {
            const int64_t strip = min(n0 / 16 + dw * kStrips + h, int64_t(a.strips) - 1), blk = strip * a.KB + kb0;
            from[h] = a.codes + blk * kBlockWords + lane * 4;
            sc[h] = reinterpret_cast<const __half2*>(a.scale + blk * per * 16) + g;
            mu[h] = a.mu ? reinterpret_cast<const __half2*>(a.mu + blk * per * 16) + g : nullptr;
        }
        if (!a.early) grid_dependency_wait();
        uint32_t next[kStrips * 2][kWords];
        __half2 sn[kStrips][kGrps], mn[kStrips][kGrps];
        auto load = [&](int i) {
#pragma unroll
            for (int h = 0; h < kStrips; ++h) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if constexpr (kTiles == 2) {
                        const uint4 u = __ldg(reinterpret_cast<const uint4*>(from[h] + i * kBlockWords + 128 * v));
                        next[2 * h + v][0] = u.x, next[2 * h + v][1] = u.y, next[2 * h + v][2] = u.z, next[2 * h + v][3] = u.w;
                    } else {
                        const uint2 u = __ldg(reinterpret_cast<const uint2*>(from[h] + (i >> 1) * kBlockWords + 128 * v + 2 * (i & 1)));
                        next[2 * h + v][0] = u.x, next[2 * h + v][1] = u.y;
                    }
                }
#pragma unroll
                for (int p = 0; p < kGrps; ++p) {
                    const int at = (kTiles == 2 ? i * per : (i >> 1) * per + (i & 1) * 64 / kGrp) + p;
                    sn[h][p] = __ldg(sc[h] + at * 8);
                    mn[h][p] = a.mu ? __ldg(mu[h] + at * 8) : __half2half2(__float2half_rn(0.f));
                }
            }
        };
        const bool swap = g & 1;
        uint32_t to[2];             // of the lane's two chunks (words 0 and 1 of a tile), row 16 kStrips dw + g
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int chunk = 4 * (swap ? 1 - e : e) + q;
            to[e] = base + uint32_t(16 * kStrips * dw + g) * 128 + uint32_t((chunk ^ g) << 4);
        }
        if (set < steps) load(set);
        int s = set % a.stages, ph = 1 ^ (set / a.stages & 1);
        for (int i = set; i < steps; i += kSets) {
            uint32_t cur[kStrips * 2][kWords];
            __half2 sv[kStrips][kGrps], mv[kStrips][kGrps];
#pragma unroll
            for (int v = 0; v < kStrips * 2; ++v)
#pragma unroll
                for (int w = 0; w < kWords; ++w) cur[v][w] = next[v][w];
#pragma unroll
            for (int h = 0; h < kStrips; ++h)
#pragma unroll
                for (int p = 0; p < kGrps; ++p) sv[h][p] = sn[h][p], mv[h][p] = mn[h][p];
            if (i + kSets < steps) load(i + kSets);
            if (i >= a.stages) ok = mbar_wait(&empty[s], ph);
            if (!ok) break;
            const uint32_t off = s * a.stage_bytes;
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int v = 0; v < kStrips * 2; ++v)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t w = (e == 0) == !swap ? cur[v][2 * j] : cur[v][2 * j + 1], w8 = w >> 8;
                        // its group of the stage: column 64 j + 32 (word)
                        constexpr int kLast = kGrps - 1;
                        const int p0 = min(64 * j / kGrp, kLast), p1 = min((64 * j + 32) / kGrp, kLast);
                        const bool second = (e == 1) != swap;
                        const __half2 sr = p0 == p1 ? sv[v >> 1][p0] : second ? sv[v >> 1][p1] : sv[v >> 1][p0];
                        const __half2 mr = p0 == p1 ? mv[v >> 1][p0] : second ? mv[v >> 1][p1] : mv[v >> 1][p0];
                        const __half2 s2 = v & 1 ? __high2half2(sr) : __low2half2(sr), m2 = v & 1 ? __high2half2(mr) : __low2half2(mr);
                        const uint4 o = make_uint4(as_u32(__hfma2(as_h2(code_pair<0, 8>(w, w8)), s2, m2)),
                                                   as_u32(__hfma2(as_h2(code_pair<1, 8>(w, w8)), s2, m2)),
                                                   as_u32(__hfma2(as_h2(code_pair<2, 8>(w, w8)), s2, m2)),
                                                   as_u32(__hfma2(as_h2(code_pair<3, 8>(w, w8)), s2, m2)));
                        sts_u4(off + to[e] + uint32_t(j * H * kABytes + v * 8 * 128), o);
                    }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
            for (s += kSets; s >= a.stages; s -= a.stages) ph ^= 1;
        }
        if (a.early) grid_dependency_wait();       // y may still be in use by the previous kernel
        // ---- epilogue
        ok = ok && mbar_wait(&done, 0);
        ok = __all_sync(0xffffffffu, ok);
        fence_after();
        if (ok) {
            // TMEM lanes 32 lq .. are this warp's (its number modulo 4 says which); the warps that share them and their half of the
            // rows take a part of the tokens each
            constexpr int kParts = kDecodeWarps / (4 * H);
            const int lq = warp & 3, half = H == 2 ? (warp - 2) >> 3 : 0, part = (warp - 2) >> 2 & (kParts - 1);
            const int cut = (a.bt / kParts + 31) / 32 * 32, c0 = part * cut, c1 = min(a.bt, c0 + cut);
            const int64_t n = n0 + half * kRowsM + lq * 32 + lane;
            const bool pairs = (a.N & 1) == 0 && !a.part;
            for (int c = c0; c < c1; c += 32) {
                uint32_t r[32];
                load_tmem32(tmem + (uint32_t(lq * 32) << 16) + uint32_t(half * 256 + c), r);
                const int64_t m = m0 + c;
                const int cnt = int(min(int64_t(min(32, c1 - c)), a.M - m));
                if (pairs) {
                    // even lanes take the even token of a pair for rows n and n + 1, odd lanes the odd one
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 1 ? r[j] : r[j + 1], 1);
                        const int mine = j + (lane & 1);
                        const __half2 v = lane & 1 ? __floats2half2_rn(__uint_as_float(got), __uint_as_float(r[j + 1]))
                                                   : __floats2half2_rn(__uint_as_float(r[j]), __uint_as_float(got));
                        if (mine < cnt && n < a.N) *reinterpret_cast<__half2*>(a.y + (m + mine) * a.N + (n & ~int64_t(1))) = v;
                    }
                } else if (n < a.N) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j < cnt) {
                            if (a.part) a.part[(int64_t(blockIdx.z) * a.M + m + j) * a.N + n] = __uint_as_float(r[j]);
                            else a.y[(m + j) * a.N + n] = __float2half_rn(__uint_as_float(r[j]));
                        }
                    }
                }
            }
        }
    }
    __syncwarp();
    if (!ok && a.status) atomicOr(a.status, kStatusTimeout);
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256 * H) : "memory");
    }
}

// ---------------------------------------------------------------- the plan of a call
struct Plan {
    int h, bt, slices, slice, stages, stage_bytes;
};

// Cycles of a call on the SMs: waves of CTAs, each 64 columns of K as long as measured for the slower of its MMAs and its
// decoding (M = 2048, 12288 x 4096: 1400 with 256 rows and tokens, 815 with 128 rows; 64 tokens: 415, decoding), about 3000 for
// a CTA's start and end; slices of K add a kernel (8000: half of that leads 400 tokens at group 32, 4096 x 4096, to slices that
// take 29.2 us against 22.1) and their sums' way through memory. At group 32 the decoding has four times
// group 128's scales to load, and chooses among them by lane, for which its variants keep a local frame of 16 or 32 bytes
// (512 tokens, 9728 x 2560: 34.8 us with 600 for it, 43.4 with 400, by the tiles it leads to; 1024 tokens, 12288 x 4096: 96.9 against 120).
Plan plan_of(const tern_nib_weight& w, int64_t M) {
    const int KB = int(w.K / kGroup);
    const int64_t sms = sm_count();
    const double decode = w.group == 32 ? 600.0 : 400.0;      // of 128 rows and 64 columns
    Plan best{};
    double least = 1e30;
    for (int h = 1; h <= 2; ++h)
        for (int bt = 32; bt <= 256; bt += 16) {
            // few tokens in one tile; many in tiles of 128 or 256 (between, the MMAs run slower: 240 200 us where 256 took 169)
            if (M > bt ? bt % 128 != 0 : bt - 16 >= M && bt > 32) continue;
            for (int slices = 1; slices <= 8 && slices <= KB; slices *= 2) {
                const int slice = (KB + slices - 1) / slices, real = (KB + slice - 1) / slice;
                const int64_t rows = (w.N + kRowsM * h - 1) / (kRowsM * h), toks = (M + bt - 1) / bt;
                const int64_t waves = (rows * toks * real + sms - 1) / sms;
                double c = double(waves) * (2.0 * slice * (h == 1 ? std::max(3.1 * bt, decode) : std::max(5.4 * bt, 1.85 * decode)) + 3000.0);
                if (real > 1) c += 8000.0 + 8.0 * double(real) * double(M) * double(w.N) / (30.0 * double(sms));
                if (c < least) {
                    least = c;
                    best = Plan{h, bt, real, slice, 0, 0};
                }
            }
        }
    best.stage_bytes = kBKs(best.h) * (best.h * kABytes + best.bt * kBK * 2);
    best.stages = std::min(kMaxStages, (kSmemMax - 2048) / best.stage_bytes);
    return best;
}

template <int kGrp, int H, int kStrips>
tern_status launch(const Plan& p, const tern_nib_weight& w, const CUtensorMap& map, Args& a, cudaStream_t stream) {
    static std::mutex mu;
    static bool configured[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TERN_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev]) {
            if (cudaFuncSetAttribute(gemm_kernel<kGrp, H, kStrips>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax - 1024) != cudaSuccess)
                return TERN_ERR_CUDA;
            configured[dev] = true;
        }
    }
    const int64_t rows = (w.N + kRowsM * H - 1) / (kRowsM * H), toks = (a.M + p.bt - 1) / p.bt;
    if (toks > 65535) return TERN_ERR_SHAPE;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows), unsigned(toks), unsigned(p.slices));
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = size_t(p.stages) * p.stage_bytes + 1024;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gemm_kernel<kGrp, H, kStrips>, map, a) == cudaSuccess ? TERN_OK : TERN_ERR_CUDA;
}

}  // namespace

namespace nib {

size_t gemm_workspace_bytes(const tern_nib_weight& w, int64_t M) {
    const Plan p = plan_of(w, M);
    return p.slices == 1 ? 0 : (size_t(p.slices) * size_t(M) * size_t(w.N) * 4 + 255) & ~size_t(255);
}

tern_status gemm_launch(const tern_nib_weight& w, const __half* x, int64_t M, __half* y, void* workspace, cudaStream_t stream) {
    const Plan p = plan_of(w, M);
    auto enc = encode_fn();
    if (!enc) return TERN_ERR_CUDA;
    CUtensorMap map;
    const cuuint64_t dims[2] = {cuuint64_t(w.K), cuuint64_t(M)};
    const cuuint64_t strides[1] = {cuuint64_t(w.K) * sizeof(__half)};
    const cuuint32_t box[2] = {kBK, cuuint32_t(p.bt)}, estr[2] = {1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(x), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return TERN_ERR_CUDA;
    Args a{};
    a.codes = w.codes;
    a.scale = reinterpret_cast<const __half*>(w.scale);
    a.mu = reinterpret_cast<const __half*>(w.mu);
    a.y = y;
    a.part = p.slices > 1 ? static_cast<float*>(workspace) : nullptr;
    a.N = w.N;
    a.M = M;
    a.KB = int(w.K / kGroup);
    a.strips = int((w.N + 15) / 16);
    a.slice = p.slice;
    a.bt = p.bt;
    a.stages = p.stages;
    a.stage_bytes = p.stage_bytes;
    a.early = (w.flags & TERN_WEIGHT_STATIC) != 0;
    a.status = async_status_word();
    auto by_group = [&](auto h, auto strips) {
        constexpr int H = decltype(h)::value, S = decltype(strips)::value;
        return w.group == 32 ? launch<32, H, S>(p, w, map, a, stream) : w.group == 64 ? launch<64, H, S>(p, w, map, a, stream)
                                                                                     : launch<128, H, S>(p, w, map, a, stream);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    // two strips per warp make four sets of warps with 128 rows (two with 256): as many stages have to fit
    const tern_status st = p.stages < 2 ? TERN_ERR_SHAPE : p.h == 2 ? by_group(Two{}, Two{}) : p.stages >= 4 ? by_group(One{}, Two{}) : by_group(One{}, One{});
    if (st != TERN_OK || p.slices == 1) return st;
    cudaError_t err;
    add_slices(a.part, p.slices, M * w.N, y, stream, err);
    return err == cudaSuccess ? TERN_OK : TERN_ERR_CUDA;
}

}  // namespace nib
}  // namespace tern
