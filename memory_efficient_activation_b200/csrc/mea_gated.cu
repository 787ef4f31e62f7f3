// mea_gated.cu -- the gated feed-forward block on the fifth-generation tensor
// cores: both projections, the activation and the product in one kernel, and
// the backward of the product in the epilogue of the matmul that feeds it.
//
//   forward:   gate = X Wg^T, up = X Wu^T (fp32 accumulation),
//              h = f(gate) up, rounded once; z = [gate | up] in bf16 where a
//              backward will need it
//   backward:  d = G Wd (fp32, never stored), from the stored z
//              dz = [d up f'(gate) | d f(gate)] and, re-populated for the
//              down projection's weight gradient, h = f(gate) up
//
// h is formed from the fp32 accumulators, not from z as stored: one rounding
// to bf16 instead of three.  The backward takes z as given.
//
// Kernel (persistent, clusters of two CTAs on two SMs, 192 threads each): as
// the plain matmul + activation, a CTA pair owns a 256-row tile whose
// accumulator has 256 columns per CTA, with the two-SM tensor-core
// instruction reading A and B from both CTAs' shared memory.
//   forward    the first CTA stages 128 rows of Wg, the second the same 128
//              rows of Wu: columns 0-127 of every accumulator row are gate,
//              columns 128-255 up of the same hidden units, so one thread
//              holds both factors of its products and nothing is exchanged.
//   backward   each CTA stages 128 columns of Wd as it is stored ([K x N], N
//              contiguous): the operand is read N-major, no transposed copy
//              of the weight is made.
// Output tiles go round-robin to CTA pairs in groups of kGroupM row tiles
// with the rows fastest, so that the pairs at work at one time share a few
// tiles of both operands in L2 (by columns alone, 64 column tiles of a 134 MB
// weight would stream from HBM once per row tile).  Every tile's sum runs
// over k in one fixed order.  Every barrier wait is bounded: one that expires
// sets g_gated_error and the roles stop issuing work.
#include <cuda_runtime.h>

#include <cstdint>

#include "mea_device.cuh"
#include "mea_gated_api.h"
#include "mea_internal.h"
#include "mea_math.cuh"
#include "mea_pipe.cuh"
#include "mea_umma.cuh"

namespace mea {

__device__ unsigned int g_gated_error = 0;

namespace {

constexpr int kBM = 256;                                    // rows of a CTA pair's tile
constexpr int kAcc = 256;                                   // accumulator columns per CTA
constexpr int kBK = 64;                                     // K per pipeline stage: 128 bytes
constexpr int kHalf = 128;                                  // rows (columns) of A and B one CTA stages
constexpr int kUmmaK = 16;
constexpr int kStages = 7;
constexpr int kThreadsG = 192;
constexpr int kGroupM = 8;                                  // row tiles per group of the tile order
constexpr uint32_t kStageA = kHalf * kBK * 2;               // 16 KB
constexpr uint32_t kStageBytes = 2 * kStageA;
constexpr uint32_t kTmemCols = 2 * kAcc;                    // 512: all of tensor memory
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + 256;

// Instruction descriptor (kind::f16): fp32 accumulator, A and B bf16, A
// K-major, B K-major (forward) or N-major (backward, bit 16), N 256, M 256.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kAcc >> 3) << 17) |
                            ((uint32_t)(kBM >> 4) << 24);
constexpr uint32_t kIdescNMajor = kIdesc | (1u << 16);

// Shared-memory descriptor of an N-major operand tile written by TMA with the
// 128-byte swizzle: each k row holds 64 contiguous elements of N (128 bytes),
// 8-row groups of k lie 1024 bytes apart (stride byte offset), and the next
// 64 elements of N lie 64 x 128 = 8192 bytes on (leading byte offset).  A K
// step of 16 advances the start address by 16 rows, 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_nmajor(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void record_error() { atomicExch(&g_gated_error, 1u); }

// Row and column tile of the t-th tile: groups of kGroupM row tiles, rows
// fastest within a group.
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int per = kGroupM * tiles_n, g = t / per, r = t - g * per;
    const int left = tiles_m - g * kGroupM, rows = left < kGroupM ? left : kGroupM;
    tn = r / rows;
    tm = g * kGroupM + r - tn * rows;
}

// 32 bf16 as 16 words, from or to a 16-byte aligned place, the first ncols (a
// multiple of 8) of them.
__device__ __forceinline__ void load32(const uint16_t *p, int ncols, uint32_t (&w)[16])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 v = 8 * q < ncols ? *(reinterpret_cast<const uint4 *>(p) + q) : make_uint4(0, 0, 0, 0);
        w[4 * q] = v.x;
        w[4 * q + 1] = v.y;
        w[4 * q + 2] = v.z;
        w[4 * q + 3] = v.w;
    }
}
__device__ __forceinline__ void store32(uint16_t *p, int ncols, const uint32_t (&w)[16])
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (8 * q < ncols)
            st_v4(reinterpret_cast<uint4 *>(p) + q, make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]));
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// r = f(v) for 32 values.
template <class A>
__device__ __forceinline__ void act32(const float (&v)[32], const Coef &k, float (&r)[32])
{
    bool tail = false;
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = A::template f<false>(v[j], k, tail);
    if (tail) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (A::is_tail(v[j], k)) r[j] = A::template f_tail<false>(v[j], k);
    }
}

// Forward epilogue of 32 hidden units of one row.
template <class A>
__device__ __forceinline__ void epilogue_fwd(const uint32_t (&ga)[32], const uint32_t (&ua)[32], const Coef &k,
                                             uint16_t *z, uint16_t *h, int64_t N, int ncols)
{
    uint32_t w[16];
    if (z) {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(__uint_as_float(ga[2 * j]), __uint_as_float(ga[2 * j + 1]));
        store32(z, ncols, w);
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(__uint_as_float(ua[2 * j]), __uint_as_float(ua[2 * j + 1]));
        store32(z + N, ncols, w);
    }
    if (h) {
        float g[32], r[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j] = __uint_as_float(ga[j]);
        act32<A>(g, k, r);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[j] = pack_bf16x2(r[2 * j] * __uint_as_float(ua[2 * j]), r[2 * j + 1] * __uint_as_float(ua[2 * j + 1]));
        store32(h, ncols, w);
    }
}

// Backward epilogue of 32 hidden units of one row.  dz may be zin.
template <class A>
__device__ __forceinline__ void epilogue_bwd(const uint32_t (&acc)[32], const Coef &k, const uint16_t *zin,
                                             uint16_t *dz, uint16_t *h, int64_t N, int ncols)
{
    uint32_t gw[16], uw[16], w[16];
    load32(zin, ncols, gw);
    load32(zin + N, ncols, uw);
    float g[32], r[32];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        g[2 * j] = lo_f(gw[j]);
        g[2 * j + 1] = hi_f(gw[j]);
    }
    act32<A>(g, k, r);
    if (h) {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(r[2 * j] * lo_f(uw[j]), r[2 * j + 1] * hi_f(uw[j]));
        store32(h, ncols, w);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
        w[j] = pack_bf16x2(r[2 * j] * __uint_as_float(acc[2 * j]), r[2 * j + 1] * __uint_as_float(acc[2 * j + 1]));
    store32(dz + N, ncols, w);
    bool tail = false;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const float d = __uint_as_float(acc[j]) * (j & 1 ? hi_f(uw[j >> 1]) : lo_f(uw[j >> 1]));
        r[j] = A::template df<false>(g[j], d, k, tail);
    }
    if (tail) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (A::template is_tail_bwd<false>(g[j], k))
                r[j] = A::template df_tail<false>(
                    g[j], __uint_as_float(acc[j]) * (j & 1 ? hi_f(uw[j >> 1]) : lo_f(uw[j >> 1])), k);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(r[2 * j], r[2 * j + 1]);
    store32(dz, ncols, w);
}

template <class A, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsG, 1)
gated_kernel(const __grid_constant__ CUtensorMap tma_x, const __grid_constant__ CUtensorMap tma_w0,
             const __grid_constant__ CUtensorMap tma_w1, int M, int N, int K, float param, const uint16_t *zin,
             uint16_t *z, uint16_t *h)
{
    constexpr int kTN = MODE == 0 ? kHalf : kAcc;          // hidden units of a tile
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);   // 1024-byte aligned tiles
    const uint32_t sbase = smem_addr(smem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);
    uint64_t *empty = full + kStages;
    uint64_t *acc_full = empty + kStages;
    uint64_t *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();          // 0: issues the MMAs of the pair
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int tiles_m = (M + kBM - 1) / kBM, tiles_n = (N + kTN - 1) / kTN;
    const int ntiles = tiles_m * tiles_n;
    const int kblocks = (K + kBK - 1) / kBK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(full + s), 1);     // the first CTA's producer; bytes of both CTAs
            mbar_init(smem_addr(empty + s), 1);    // one commit from the first CTA
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(acc_full + b), 1);
            mbar_init(smem_addr(acc_empty + b), 8); // four epilogue warps of each CTA
        }
        mbar_init_fence();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();                                // barriers of both CTAs initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs) {
                int tm, tn;
                tile_of(t, tiles_m, tiles_n, tm, tn);
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const int s = it % kStages, round = it / kStages;
                    if (round > 0 && !mbar_wait(smem_addr(empty + s), (round & 1) ^ 1)) {
                        record_error();
                        ok = false;
                        break;
                    }
                    const uint32_t fb = cluster_addr(smem_addr(full + s), 0);
                    if (rank == 0) mbar_arrive_expect_tx(smem_addr(full + s), 2 * kStageBytes);
                    const uint32_t sa = sbase + s * kStageBytes, sb = sa + kStageA;
                    tma_load_2d_pair(sa, &tma_x, kb * kBK, tm * kBM + rank * kHalf, fb);
                    if constexpr (MODE == 0) {
                        tma_load_2d_pair(sb, rank == 0 ? &tma_w0 : &tma_w1, kb * kBK, tn * kTN, fb);
                    } else {
                        // two boxes of 64 k rows x 64 columns of Wd
                        const int c = tn * kTN + rank * kHalf;
                        tma_load_2d_pair(sb, &tma_w0, c, kb * kBK, fb);
                        tma_load_2d_pair(sb + kStageA / 2, &tma_w0, c + 64, kb * kBK, fb);
                    }
                }
            }
            // every load issued has landed before teardown: this CTA's stages
            // are released (empty) once the MMAs that read them complete
            for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
                if (!mbar_wait(smem_addr(empty + j % kStages), (j / kStages) & 1)) record_error();
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int it = 0, lt = 0;
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs, ++lt) {
                const int b = lt & 1, use = lt >> 1;
                if (use > 0 && !mbar_wait(smem_addr(acc_empty + b), (use & 1) ^ 1)) {
                    record_error();
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + b * kAcc;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(smem_addr(full + s), (it / kStages) & 1)) {
                        record_error();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = sbase + s * kStageBytes, sb = sa + kStageA;
#pragma unroll
                    for (int k = 0; k < kBK / kUmmaK; ++k) {
                        const uint64_t da = sdesc_sw128(sa + k * kUmmaK * 2);
                        if constexpr (MODE == 0)
                            umma_bf16_pair(d, da, sdesc_sw128(sb + k * kUmmaK * 2), kIdesc, (kb | k) != 0);
                        else
                            umma_bf16_pair(d, da, sdesc_nmajor(sb + k * kUmmaK * 128), kIdescNMajor, (kb | k) != 0);
                    }
                    umma_commit_pair(smem_addr(empty + s));
                }
                if (ok) umma_commit_pair(smem_addr(acc_full + b));
            }
        }
        __syncwarp();
    } else {
        // epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. + 31 of
        // this CTA, i.e. rows rank * 128 + 32 (w % 4) + lane of the tile
        const int q = warp & 3;
        const Coef k = A::coef(param);
        const uint32_t release = cluster_addr(smem_addr(acc_empty), 0);
        int lt = 0;
        for (int t = pair; t < ntiles; t += npairs, ++lt) {
            const int b = lt & 1, use = lt >> 1;
            if (!mbar_wait(smem_addr(acc_full + b), use & 1)) {
                record_error();
                break;
            }
            tc_fence_after();
            int tm, tn;
            tile_of(t, tiles_m, tiles_n, tm, tn);
            const int row = tm * kBM + (int)rank * kHalf + q * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + b * kAcc;
#pragma unroll 1
            for (int c = 0; c < kTN / 32; ++c) {
                uint32_t v[32], u[32];
                tmem_ld32(lanes + c * 32, v);
                if constexpr (MODE == 0) tmem_ld32(lanes + kHalf + c * 32, u);
                const int col = tn * kTN + c * 32;
                if (row < M && col < N) {
                    const int ncols = N - col < 32 ? N - col : 32;
                    const int64_t oz = (int64_t)row * 2 * N + col, oh = (int64_t)row * N + col;
                    if constexpr (MODE == 0)
                        epilogue_fwd<A>(v, u, k, z ? z + oz : nullptr, h ? h + oh : nullptr, N, ncols);
                    else
                        epilogue_bwd<A>(v, k, zin + oz, z + oz, h ? h + oh : nullptr, N, ncols);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(release + 8 * b);
        }
    }
    pdl_trigger();
    tc_fence_before();
    cluster_sync();                                // no CTA leaves while its pair may touch its memory
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ------------------------------------------------------------ host side

template <class A, int MODE>
cudaError_t launch_one(const GatedLaunch &a)
{
    CUtensorMap mx, mw0, mw1;
    bool ok = bf16_tile_map(&mx, a.x, a.M, a.K, kHalf);
    if (MODE == 0) {
        ok = ok && bf16_tile_map(&mw0, a.w0, a.N, a.K, kHalf) && bf16_tile_map(&mw1, a.w1, a.N, a.K, kHalf);
    } else {
        ok = ok && bf16_tile_map(&mw0, a.w0, a.K, a.N, kBK);
        mw1 = mw0;
    }
    if (!ok) return cudaErrorInvalidValue;
    auto kernel = gated_kernel<A, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    const int tn = MODE == 0 ? kHalf : kAcc;
    const int64_t tiles = ((a.M + kBM - 1) / kBM) * ((a.N + tn - 1) / tn);
    const int pairs_max = sm_count() / 2;
    const int pairs = (int)(tiles < pairs_max ? tiles : pairs_max);
    return launch_pdl(kernel, dim3((unsigned)(2 * pairs)), dim3(kThreadsG), kSmemBytes, a.stream, mx, mw0, mw1,
                      (int)a.M, (int)a.N, (int)a.K, a.param, static_cast<const uint16_t *>(a.zin),
                      static_cast<uint16_t *>(a.z), static_cast<uint16_t *>(a.h));
}

template <int MODE>
cudaError_t by_act(const GatedLaunch &a)
{
    switch (a.act) {
    case 0: return launch_one<ReLU, MODE>(a);
    case 1: return launch_one<LeakyReLU, MODE>(a);
    case 2: return launch_one<Sigmoid, MODE>(a);
    case 3: return launch_one<Tanh, MODE>(a);
    case 4: return launch_one<GeluErf, MODE>(a);
    case 5: return launch_one<GeluTanh, MODE>(a);
    case 6: return launch_one<Swish, MODE>(a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t gated_error_word(int clear, unsigned int *word)
{
    cudaError_t e = cudaMemcpyFromSymbol(word, g_gated_error, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_gated_error, &zero, sizeof(unsigned int));
    }
    return e;
}

cudaError_t launch_gated(const GatedLaunch &a) { return a.mode == 0 ? by_act<0>(a) : by_act<1>(a); }

}  // namespace mea
