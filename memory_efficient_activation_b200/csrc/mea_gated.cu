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
// The plain products around the block (h Wd^T, dz [Wg; Wu], dz^T X, G^T h) run
// on the same kernel, each operand read as it is stored.
//
// Kernel (persistent, clusters of two CTAs on two SMs, four or eight epilogue
// warps beside the loading and the issuing one): as the plain matmul + activation, a CTA pair owns a 256-row tile whose
// accumulator has 256 columns per CTA, with the two-SM tensor-core
// instruction reading A and B from both CTAs' shared memory.
//   forward    the first CTA stages 128 rows of Wg, the second the same 128
//              rows of Wu: columns 0-127 of every accumulator row are gate,
//              columns 128-255 up of the same hidden units, so one thread
//              holds both factors of its products and nothing is exchanged.
//   backward   each CTA stages 128 columns of Wd as it is stored ([K x N], N
//              contiguous): the operand is read N-major, no transposed copy
//              of the weight is made.
// Output tiles go round-robin to CTA pairs in groups of 8 or 16 row tiles
// with the rows fastest, so that the pairs at work at one time share a few
// tiles of both operands in L2 (by columns alone, 64 column tiles of a 134 MB
// weight would stream from HBM once per row tile).  Every tile's sum runs
// over k in one fixed order.  Every barrier wait is bounded: one that expires
// sets g_gated_error and the roles stop issuing work.
//
// Measured, bf16, swish, [8192 x 4096] and 8192 hidden units.  One launch at
// full clocks: forward with z 687 us (1.60 PFLOP/s; tensor pipe 90% active),
// backward 390 (1.41; 75%).  Back to back, under the board's power limit:
// forward 785-815 (1.35-1.40, as a library's plain product of that size
// there), backward 465-500 (1.10-1.18).  What the backward lacks is L2 and
// shared-memory bandwidth: z, dz and h are 10 bytes per element of an output
// that the operands' tiles already stream 128 FLOP per byte for (without its
// stores 375 us, without loads, stores and arithmetic 339, one launch each).
#include <cuda_runtime.h>

#include <cmath>
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

// What a kernel computes: the two passes of the gated block, or the plain
// product C = op(A) op(B)^T around it, with A stored [M x K] or [K x M] and B
// stored [N x K] or [K x N].
enum Mode { kFwd, kBwd, kPlainNT, kPlainNN, kPlainTN };

constexpr int kBM = 256;                                    // rows of a CTA pair's tile
constexpr int kAcc = 256;                                   // accumulator columns per CTA
constexpr int kBK = 64;                                     // K per pipeline stage: 128 bytes
constexpr int kHalf = 128;                                  // rows (columns) of A and B one CTA stages
constexpr int kUmmaK = 16;
constexpr uint32_t kStageA = kHalf * kBK * 2;               // 16 KB
constexpr uint32_t kStageBytes = 2 * kStageA;
constexpr uint32_t kTmemCols = 2 * kAcc;                    // 512: all of tensor memory

// Epilogue chunk: a warp's 32 rows x 32 columns of one tensor, 64 bytes per
// row in shared memory under the 64-byte swizzle, moved by TMA.
constexpr uint32_t kChunk = 32 * 32 * 2;

// EW: epilogue warps, four (one per quarter of tensor memory) or eight (each
// half of the columns too).  Four, with more pipeline stages, where a pair of
// SMs has several tiles and the epilogue of one runs beside the matmul of the
// next; eight where it has one and nothing hides the epilogue.
template <Mode MODE, int EW>
struct Shape {
    static constexpr bool kMMajorA = MODE == kPlainTN;
    static constexpr bool kNMajorB = MODE == kBwd || MODE == kPlainNN || MODE == kPlainTN;
    static constexpr int kTN = MODE == kFwd ? kHalf : kAcc;              // output columns of a tile
    // Row tiles per group of the tile order, measured back to back under the
    // power limit: 16 for the forward ([8192 x 2 x 8192 x 4096] 831 us against
    // 844 at 8 and 883 at 4), 8 elsewhere (backward 498; 508 at 16, 523 at 4).
    static constexpr int kGroupM = MODE == kFwd ? 16 : 8;
    static constexpr int kWarps = EW;
    static constexpr int kThreads = 64 + 32 * kWarps;
    // Chunk buffers per warp.  Backward: gate and up as they arrive (read into
    // registers at once, so that the next are on their way during the
    // arithmetic; of two chunks with four warps, 32 KB in flight per SM),
    // dgate, dup and h.  Forward: gate, up and h; a second set of them would
    // cost a pipeline stage (157 against 163 us at [4096 x 2 x 5464 x 2048]).
    // Plain: C in turn.
    static constexpr int kIn = MODE == kBwd ? 8 / EW : 0;
    static constexpr int kOut = MODE == kBwd || MODE == kFwd ? 1 : 4;
    static constexpr int kChunks = MODE == kBwd ? 2 * kIn + 3 : MODE == kFwd ? 3 : kOut;
    static constexpr uint32_t kEpiBytes = kWarps * kChunks * kChunk;
    // Pipeline stages: what is left of the shared memory.
    static constexpr int kStages = MODE == kBwd ? (EW == 8 ? 4 : 5) : 6;
    static constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + kEpiBytes + 256;
    static_assert(kSmemBytes <= 232448, "shared memory of a block");
};

// Instruction descriptor (kind::f16): fp32 accumulator, A and B bf16, M 256;
// A K-major or M-major (bit 15), B K-major or N-major (bit 16), N / 8 from bit
// 17 on.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kBM >> 4) << 24);

__device__ __forceinline__ void record_error() { atomicExch(&g_gated_error, 1u); }

// Row and column tile of the t-th tile: groups of GM row tiles, rows fastest
// within a group.
template <int GM>
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int per = GM * tiles_n, g = t / per, r = t - g * per;
    const int left = tiles_m - g * GM, rows = left < GM ? left : GM;
    tn = r / rows;
    tm = g * GM + r - tn * rows;
}

// Row `lane` of a chunk in shared memory, 32 bf16 as 16 words.  The 64-byte
// swizzle exchanges the 16-byte quarters of a row by bits 1-2 of its number,
// so a warp's accesses touch every bank once per quarter.
__device__ __forceinline__ uint32_t chunk_quarter(uint32_t chunk, int lane, int q)
{
    return chunk + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4);
}
__device__ __forceinline__ void load_row(uint32_t chunk, int lane, uint32_t (&w)[16])
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * q]), "=r"(w[4 * q + 1]), "=r"(w[4 * q + 2]), "=r"(w[4 * q + 3])
                     : "r"(chunk_quarter(chunk, lane, q))
                     : "memory");
}
__device__ __forceinline__ void store_row(uint32_t chunk, int lane, const uint32_t (&w)[16])
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(chunk_quarter(chunk, lane, q)), "r"(w[4 * q]),
                     "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                     : "memory");
}

// TMA copies of a chunk: this CTA's shared memory to and from [row x col].
__device__ __forceinline__ void chunk_load(uint32_t dst, const CUtensorMap *map, int col, int row, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void chunk_store(const CUtensorMap *map, int col, int row, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread's stores have read their source.
template <int N>
__device__ __forceinline__ void store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// This thread's writes to shared memory become visible to TMA.
__device__ __forceinline__ void fence_to_tma() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

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

// Forward: h = f(gate) up of 32 hidden units of one row, in words.
template <class A>
__device__ __forceinline__ void product_fwd(const uint32_t (&ga)[32], const uint32_t (&ua)[32], const Coef &k,
                                            uint32_t (&w)[16])
{
    float g[32], r[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] = __uint_as_float(ga[j]);
    act32<A>(g, k, r);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        w[j] = pack_bf16x2(r[2 * j] * __uint_as_float(ua[2 * j]), r[2 * j + 1] * __uint_as_float(ua[2 * j + 1]));
}

__device__ __forceinline__ void pack32(const uint32_t (&a)[32], uint32_t (&w)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
}

// f and f' of two values from one set of exponentials and reciprocals, in
// packed pairs: the backward needs both of every element.  `tail` is set where
// either leaves its main path; the elements that is_tail (f) and is_tail_bwd
// (f') name are then taken again in scalar form.
template <class A>
struct Both {
    static __device__ __forceinline__ void eval(float x0, float x1, const Coef &k, bool &tail, F2 &f, F2 &df)
    {
        f = pk(A::template f<false>(x0, k, tail), A::template f<false>(x1, k, tail));
        df = pk(A::template df<false>(x0, 1.f, k, tail), A::template df<false>(x1, 1.f, k, tail));
    }
};
// s = 1 / (1 + E), E = 2^t: f = x s, f' = s (1 + alpha x E s), E s = Sigmoid(-alpha x);
// alpha x is limited as in df, so that an infinite one times E = 0 stays 0.
template <bool RC>
struct Both<SwishT<RC>> {
    static __device__ __forceinline__ void eval(float x0, float x1, const Coef &k, bool &tail, F2 &f, F2 &df)
    {
        const F2 x = pk(x0, x1);
        float t0, t1, a0, a1, z0, z1;
        upk(mul2(x, sp2(k.c_hi)), t0, t1);
        upk(mul2(x, sp2(k.p)), z0, z1);
        const F2 E = pk(ex2_ftz(t0), ex2_ftz(t1));
        tail |= fmaxf(t0, t1) > kTailT;
        if constexpr (RC)
            tail |= fminf(fabsf(__fsub_rn(t0, SwishT<RC>::kRootT)), fabsf(__fsub_rn(t1, SwishT<RC>::kRootT))) <
                    SwishT<RC>::kRootWinT;
        upk(add2(E, sp2(1.f)), a0, a1);
        const F2 s = pk(rcp_ftz(a0), rcp_ftz(a1));
        f = mul2(x, s);
        df = mul2(s, fma2(pk(fminf(z0, kBig), fminf(z1, kBig)), mul2(E, s), sp2(1.f)));
    }
};
// The same with t a cubic and x v' for alpha x (x beyond 2e10 in size, where
// x v' could overflow, is tail on the positive side by t < -kHugeT).
template <>
struct Both<GeluTanh> {
    static __device__ __forceinline__ void eval(float x0, float x1, const Coef &, bool &tail, F2 &f, F2 &df)
    {
        const F2 x = pk(x0, x1), x2 = mul2(x, x);
        float t0, t1, a0, a1;
        upk(mul2(x, fma2(sp2(GeluTanh::kC3f), x2, sp2(GeluTanh::kC1f))), t0, t1);
        const F2 E = pk(ex2_ftz(t0), ex2_ftz(t1));
        tail |= (fmaxf(t0, t1) > kTailT) | (fminf(t0, t1) < -GeluTanh::kHugeT);
        upk(add2(E, sp2(1.f)), a0, a1);
        const F2 s = pk(rcp_ftz(a0), rcp_ftz(a1));
        f = mul2(x, s);
        const F2 q = mul2(x, fma2(sp2(GeluTanh::kK3x3f), x2, sp2(GeluTanh::kK1f)));
        df = mul2(s, fma2(q, mul2(E, s), sp2(1.f)));
    }
};
// Phi(x) by the backward's erfc (one Gaussian for it and for x phi(x)).
template <>
struct Both<GeluErf> {
    static __device__ __forceinline__ void eval(float x0, float x1, const Coef &, bool &tail, F2 &f, F2 &df)
    {
        const F2 x = pk(x0, x1), w = mul2(x, sp2(GeluErf::kNegRsqrt2Hi));
        float w0, w1, d0, d1, v0, v1, a0, a1;
        upk(w, w0, w1);
        upk(add2(pk(fabsf(w0), fabsf(w1)), sp2(2.0f)), d0, d1);
        const F2 h = pk(rcp_ftz(d0), rcp_ftz(d1));
        upk(mul2(mul2(w, w), sp2(-GeluErf::kLog2ef)), v0, v1);
        tail |= fminf(x0, x1) < GeluErf::kTailX;
        const F2 g = pk(ex2_ftz(v0), ex2_ftz(v1));
        upk(mul2(mul2(h, GeluErf::q8_2(h)), g), a0, a1);
        const F2 phi = pk(w0 >= 0.f ? a0 : 1.f - a0, w1 >= 0.f ? a1 : 1.f - a1);
        f = mul2(x, phi);
        df = fma2(mul2(x, sp2(GeluErf::kRsqrt2Pi)), g, phi);
    }
};

__device__ __forceinline__ uint32_t pack_f2(F2 v)
{
    float a, b;
    upk(v, a, b);
    return pack_bf16x2(a, b);
}

// One element again, where it may have left the main path: e its place in the
// pair (0 low, 1 high).
template <class A>
__device__ __forceinline__ void bwd_again(uint32_t gw, uint32_t uw, float d, int e, const Coef &k, float &dg, float &du,
                                          float &h)
{
    const float g = e ? hi_f(gw) : lo_f(gw), u = e ? hi_f(uw) : lo_f(uw);
    if (A::is_tail(g, k)) {
        const float f = A::template f_tail<false>(g, k);
        du = f * d;
        h = f * u;
    }
    if (A::template is_tail_bwd<false>(g, k)) dg = A::template df_tail<false>(g, d * u, k);
}

// Backward of 32 hidden units of one row: gw, uw the stored gate and up, in
// place of which dgate and dup are returned; hw the product.
template <class A>
__device__ __forceinline__ void product_bwd(const uint32_t (&acc)[32], const Coef &k, uint32_t (&gw)[16],
                                            uint32_t (&uw)[16], uint32_t (&hw)[16])
{
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        uint32_t dg[8], du[8];
        bool tail = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = 8 * p + j;
            const F2 u = pk(lo_f(uw[i]), hi_f(uw[i]));
            const F2 d = pk(__uint_as_float(acc[2 * i]), __uint_as_float(acc[2 * i + 1]));
            F2 f, df;
            Both<A>::eval(lo_f(gw[i]), hi_f(gw[i]), k, tail, f, df);
            hw[i] = pack_f2(mul2(f, u));
            du[j] = pack_f2(mul2(f, d));
            dg[j] = pack_f2(mul2(mul2(d, u), df));
        }
        if (tail) {
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 8 * p + j;
                    float vg = e ? hi_f(dg[j]) : lo_f(dg[j]), vu = e ? hi_f(du[j]) : lo_f(du[j]),
                          vh = e ? hi_f(hw[i]) : lo_f(hw[i]);
                    bwd_again<A>(gw[i], uw[i], __uint_as_float(e ? acc[2 * i + 1] : acc[2 * i]), e, k, vg, vu, vh);
                    dg[j] = e ? pack_bf16x2(lo_f(dg[j]), vg) : pack_bf16x2(vg, hi_f(dg[j]));
                    du[j] = e ? pack_bf16x2(lo_f(du[j]), vu) : pack_bf16x2(vu, hi_f(du[j]));
                    hw[i] = e ? pack_bf16x2(lo_f(hw[i]), vh) : pack_bf16x2(vh, hi_f(hw[i]));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            gw[8 * p + j] = dg[j];
            uw[8 * p + j] = du[j];
        }
    }
}

// Tensor maps of a launch.  Forward: x, w0 = Wg, w1 = Wu, out0 and out1 the
// halves of z, out2 = h.  Backward: x = G, w0 = Wd, in0 and in1 the halves of
// the stored z, out0 and out1 those of dz, out2 = h.  Plain: x = A, w0 = B,
// out0 = C.
struct Maps {
    CUtensorMap x, w0, w1, in0, in1, out0, out1, out2;
};

template <class A, Mode MODE, int EW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<MODE, EW>::kThreads, 1)
gated_kernel(const __grid_constant__ Maps maps, int M, int N, int K, int tw, float param, int want01, int want2)
{
    using S = Shape<MODE, EW>;
    constexpr int kTN = S::kTN, kStages = S::kStages;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);   // 1024-byte aligned tiles
    const uint32_t sbase = smem_addr(smem);
    const uint32_t ebase = sbase + kStages * kStageBytes;  // epilogue chunks
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes + S::kEpiBytes);
    uint64_t *empty = full + kStages;
    uint64_t *acc_full = empty + kStages;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *in_full = acc_empty + 2;                     // backward: a chunk of z has landed, two per warp
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(in_full + 2 * S::kWarps);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();          // 0: issues the MMAs of the pair
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int tiles_m = (M + kBM - 1) / kBM, tiles_n = (N + tw - 1) / tw;
    const int ntiles = tiles_m * tiles_n;
    const int kblocks = (K + kBK - 1) / kBK;

    if (threadIdx.x == 32) {                       // descriptors on their way while the barriers are set up
        prefetch_map(&maps.x);
        prefetch_map(&maps.w0);
        if constexpr (MODE == kFwd) prefetch_map(&maps.w1);
        if constexpr (MODE == kBwd) {
            prefetch_map(&maps.in0);
            prefetch_map(&maps.in1);
        }
        if (MODE != kFwd || want01) prefetch_map(&maps.out0);
        if constexpr (MODE == kFwd || MODE == kBwd) {
            if (want01) prefetch_map(&maps.out1);
            if (want2) prefetch_map(&maps.out2);
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(full + s), 1);     // the first CTA's producer; bytes of both CTAs
            mbar_init(smem_addr(empty + s), 1);    // one commit from the first CTA
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(acc_full + b), 1);
            mbar_init(smem_addr(acc_empty + b), 2 * S::kWarps);   // the epilogue warps of both CTAs
        }
        for (int i = 0; i < 2 * S::kWarps; ++i) mbar_init(smem_addr(in_full + i), 1);
        mbar_init_fence();
    }
    if (warp == 1) {
        __syncwarp();
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
                tile_of<S::kGroupM>(t, tiles_m, tiles_n, tm, tn);
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
                    const int ra = tm * kBM + rank * kHalf;
                    if constexpr (S::kMMajorA) {
                        // two boxes of 64 k rows x 64 elements of M
                        tma_load_2d_pair(sa, &maps.x, ra, kb * kBK, fb);
                        tma_load_2d_pair(sa + kStageA / 2, &maps.x, ra + 64, kb * kBK, fb);
                    } else {
                        tma_load_2d_pair(sa, &maps.x, kb * kBK, ra, fb);
                    }
                    if constexpr (MODE == kFwd) {
                        tma_load_2d_pair(sb, rank == 0 ? &maps.w0 : &maps.w1, kb * kBK, tn * tw, fb);
                    } else {
                        const int c = tn * tw + (int)rank * (tw / 2);
                        if constexpr (S::kNMajorB) {
                            tma_load_2d_pair(sb, &maps.w0, c, kb * kBK, fb);
                            tma_load_2d_pair(sb + kStageA / 2, &maps.w0, c + 64, kb * kBK, fb);
                        } else {
                            tma_load_2d_pair(sb, &maps.w0, kb * kBK, c, fb);
                        }
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
            const uint32_t idesc = kIdesc | (S::kMMajorA ? 1u << 15 : 0u) | (S::kNMajorB ? 1u << 16 : 0u) |
                                   ((uint32_t)((MODE == kFwd ? 2 * tw : tw) >> 3) << 17);
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
                        const uint64_t da = S::kMMajorA ? sdesc_mn(sa + k * kUmmaK * 128) : sdesc_sw128(sa + k * kUmmaK * 2);
                        const uint64_t db = S::kNMajorB ? sdesc_mn(sb + k * kUmmaK * 128) : sdesc_sw128(sb + k * kUmmaK * 2);
                        umma_bf16_pair(d, da, db, idesc, (kb | k) != 0);
                    }
                    umma_commit_pair(smem_addr(empty + s));
                }
                if (ok) umma_commit_pair(smem_addr(acc_full + b));
            }
        }
        __syncwarp();
    } else {
        // epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. + 31 of
        // this CTA, i.e. rows rank * 128 + 32 (w % 4) + lane of the tile, in
        // chunks of 32 columns.  Results (and the backward's z) pass through
        // the warp's own chunk buffers, moved by TMA: a thread owns a row, and
        // 16-byte accesses of 32 rows straight to global memory took 32
        // cache lines an instruction, more time than the matmul at K 2048.
        const int q = warp & 3, ew = warp - 2;
        const Coef k = A::coef(param);
        const uint32_t release = cluster_addr(smem_addr(acc_empty), 0);
        const uint32_t mine = ebase + ew * (S::kChunks * kChunk);
        constexpr int kIn = S::kIn > 0 ? S::kIn : 1;
        constexpr int kHalves = S::kWarps / 4, kMost = kTN / 32 / kHalves;   // column shares, chunks of one
        const int c0 = (ew >> 2) * kMost;                  // this warp's first chunk
        const uint32_t in_bars = smem_addr(in_full + 2 * ew);
        const int row_in = (int)rank * kHalf + q * 32;
        // Where this warp's chunks of tile t lie, and how many have something
        // in them.  Its divisions are done once per tile: once per chunk they
        // took as long as the arithmetic.
        struct Place {
            int row, col, nc;
        };
        auto place = [&](int t) {
            int tm, tn;
            tile_of<S::kGroupM>(t, tiles_m, tiles_n, tm, tn);
            Place p;
            p.row = tm * kBM + row_in;
            p.col = tn * tw + c0 * 32;
            const int end = tn * tw + tw < N ? tn * tw + tw : N, left = (end - p.col + 31) / 32;
            p.nc = p.row >= M || left < 0 ? 0 : left < kMost ? left : kMost;
            return p;
        };
        // backward: z of chunk fc of the tile at fp (the ft-th), the next one
        // to fetch; fetched counts those asked for
        int ft = pair, fc = 0, fetched = 0;
        Place fp = place(ft);
        auto seek = [&] {                                  // the next tile with chunks
            while (ft < ntiles && fp.nc == 0) {
                ft += npairs;
                if (ft < ntiles) fp = place(ft);
            }
        };
        auto fetch = [&] {
            if (ft >= ntiles) return;
            if (lane == 0) {
                const uint32_t k = fetched % kIn, dst = mine + k * 2 * kChunk, bar = in_bars + 8 * k;
                mbar_arrive_expect_tx(bar, 2 * kChunk);
                chunk_load(dst, &maps.in0, fp.col + fc * 32, fp.row, bar);
                chunk_load(dst + kChunk, &maps.in1, fp.col + fc * 32, fp.row, bar);
            }
            ++fetched;
            if (++fc == fp.nc) {
                fc = 0;
                fp.nc = 0;
                seek();
            }
        };
        int n = 0;                                         // chunks taken so far
        bool ok = true;
        if constexpr (MODE == kBwd) {
            seek();
            for (int i = 0; i < kIn; ++i) fetch();
        }
        int lt = 0;
        for (int t = pair; t < ntiles; t += npairs, ++lt) {
            const int b = lt & 1, use = lt >> 1;
            if (!mbar_wait(smem_addr(acc_full + b), use & 1)) {
                record_error();
                ok = false;
            }
            if (!ok) break;
            tc_fence_after();
            const Place p = place(t);
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + b * kAcc;
#pragma unroll 1
            for (int c = 0; c < p.nc; ++c, ++n) {
                uint32_t v[32], w[16];
                tmem_ld32(lanes + (c0 + c) * 32, v);
                const int row = p.row, col = p.col + c * 32;
                const uint32_t buf = mine + (MODE == kBwd ? 2 * kIn : n % S::kOut) * kChunk;
                if constexpr (MODE == kFwd) {
                    uint32_t u[32];
                    tmem_ld32(lanes + tw + (c0 + c) * 32, u);
                    if (lane == 0) store_wait_read<S::kOut - 1>();
                    __syncwarp();
                    if (want01) {
                        pack32(v, w);
                        store_row(buf, lane, w);
                        pack32(u, w);
                        store_row(buf + kChunk, lane, w);
                    }
                    if (want2) {
                        product_fwd<A>(v, u, k, w);
                        store_row(buf + 2 * kChunk, lane, w);
                    }
                } else if constexpr (MODE == kBwd) {
                    uint32_t uw[16], hw[16];
                    const uint32_t in = mine + n % kIn * 2 * kChunk;
                    if (!mbar_wait(in_bars + 8 * (n % kIn), (n / kIn) & 1)) {
                        record_error();
                        ok = false;
                        break;
                    }
                    load_row(in, lane, w);
                    load_row(in + kChunk, lane, uw);
                    __syncwarp();
                    fetch();
                    product_bwd<A>(v, k, w, uw, hw);
                    if (lane == 0) store_wait_read<0>();   // of the chunk before: long done
                    __syncwarp();
                    store_row(buf, lane, w);
                    store_row(buf + kChunk, lane, uw);
                    if (want2) store_row(buf + 2 * kChunk, lane, hw);
                } else {
                    pack32(v, w);
                    if (lane == 0) store_wait_read<S::kOut - 1>();
                    __syncwarp();
                    store_row(buf, lane, w);
                }
                fence_to_tma();
                __syncwarp();
                if (lane == 0) {
                    if (MODE != kFwd || want01) chunk_store(&maps.out0, col, row, buf);
                    if constexpr (MODE == kFwd || MODE == kBwd) {
                        if (want01) chunk_store(&maps.out1, col, row, buf + kChunk);
                        if (want2) chunk_store(&maps.out2, col, row, buf + 2 * kChunk);
                    }
                    store_commit();
                }
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(release + 8 * b);
        }
        // what is in flight has landed before this CTA's memory goes away
        for (; n < fetched; ++n)
            if (!mbar_wait(in_bars + 8 * (n % kIn), (n / kIn) & 1)) record_error();
        if (lane == 0) store_wait_read<0>();
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

// 2-D map of one [rows x cols] bf16 tensor with row stride ld (elements) for
// the epilogue's chunks: box of 32 x 32, 64-byte swizzle.
bool chunk_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld)
{
    return bf16_map(map, base, rows, cols, ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

template <class A, Mode MODE, int EW>
cudaError_t launch_warps(const GatedLaunch &a, const Maps &m, int tw, int pairs)
{
    using S = Shape<MODE, EW>;
    auto kernel = gated_kernel<A, MODE, EW>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)(2 * pairs)), dim3(S::kThreads), S::kSmemBytes, a.stream, m, (int)a.M,
                      (int)a.N, (int)a.K, tw, a.param, (int)(a.z != nullptr), (int)(a.h != nullptr));
}

template <class A, Mode MODE>
cudaError_t launch_one(const GatedLaunch &a)
{
    using S = Shape<MODE, 4>;
    Maps m;
    // an operand stored with K contiguous: boxes of 128 rows x 64 k; one with
    // M or N contiguous: boxes of 64 k x 64
    bool ok = S::kMMajorA ? bf16_tile_map(&m.x, a.x, a.K, a.M, kBK) : bf16_tile_map(&m.x, a.x, a.M, a.K, kHalf);
    ok = ok && (S::kNMajorB ? bf16_tile_map(&m.w0, a.w0, a.K, a.N, kBK) : bf16_tile_map(&m.w0, a.w0, a.N, a.K, kHalf));
    m.w1 = m.in0 = m.in1 = m.out0 = m.out1 = m.out2 = m.w0;
    const uint16_t *zin = static_cast<const uint16_t *>(a.zin);
    uint16_t *z = static_cast<uint16_t *>(a.z);
    if (MODE == kFwd) ok = ok && bf16_tile_map(&m.w1, a.w1, a.N, a.K, kHalf);
    if (MODE == kBwd)
        ok = ok && chunk_map(&m.in0, zin, a.M, a.N, 2 * a.N) && chunk_map(&m.in1, zin + a.N, a.M, a.N, 2 * a.N);
    if (MODE == kFwd || MODE == kBwd) {
        if (z) ok = ok && chunk_map(&m.out0, z, a.M, a.N, 2 * a.N) && chunk_map(&m.out1, z + a.N, a.M, a.N, 2 * a.N);
        if (a.h) ok = ok && chunk_map(&m.out2, a.h, a.M, a.N, a.N);
    } else {
        ok = ok && chunk_map(&m.out0, z, a.M, a.N, a.N);
    }
    if (!ok) return cudaErrorInvalidValue;
    // Tiles of 224 columns instead of 256 where they take no more rounds of all
    // pairs (us back to back, 224 / 256: plain [1024 x 1024 x 1024] 8.5 / 9.0,
    // G^T h of 2048 x 5464 and 4096 tokens, three rounds, 71 / 75; the backward
    // [1023 x 2728 x 1024] 15.7 / 17.1, [1024 x 1024 x 1024] 13.9 / 15.2).
    // With a round more they lose, although its columns are fewer: the operands
    // are read more often ([8192 x 5464 x 1024], 11 rounds against 10, plain 86 /
    // 76, backward 173 / 171).  The operand's tile in shared memory keeps its
    // size, its last columns are loaded for nothing.
    // Not in the forward, where 112 hidden units took as long as 128: loads
    // out of L2 bound it there.
    const int pairs = sm_count() / 2;
    const int64_t rows = (a.M + kBM - 1) / kBM;
    auto rounds = [&](int64_t w) { return (rows * ((a.N + w - 1) / w) + pairs - 1) / pairs; };
    const int tw = MODE != kFwd && rounds(S::kTN - 32) <= rounds(S::kTN) ? S::kTN - 32 : S::kTN;
    const int64_t tiles = rows * ((a.N + tw - 1) / tw);
    // The forward and the plain products, whose epilogue does little, gained
    // nothing from eight warps; the backward 7 to 14 percent (back to back,
    // [1023 x 2728 x 1024] 16.9 -> 15.7 us, [300 x 2048 x 512] 13.6 -> 11.7).
    if constexpr (MODE == kBwd)
        if (tiles <= pairs) return launch_warps<A, MODE, 8>(a, m, tw, (int)tiles);
    return launch_warps<A, MODE, 4>(a, m, tw, (int)(tiles < pairs ? tiles : pairs));
}

template <Mode MODE>
cudaError_t by_act(const GatedLaunch &a)
{
    switch (a.act) {
    case 0: return launch_one<ReLU, MODE>(a);
    case 1: return launch_one<LeakyReLU, MODE>(a);
    case 2: return launch_one<Sigmoid, MODE>(a);
    case 3: return launch_one<Tanh, MODE>(a);
    case 4: return launch_one<GeluErf, MODE>(a);
    case 5: return launch_one<GeluTanh, MODE>(a);
    case 6: {
        // f alone has no zero of f' to guard, nor has f' where alpha is a power
        // of two: bf16 inputs then keep their distance from it
        int e;
        const bool pow2 = a.param == 0.f || fabsf(frexpf(a.param, &e)) == 0.5f;
        return MODE == kFwd || pow2 ? launch_one<SwishT<false>, MODE>(a) : launch_one<SwishT<true>, MODE>(a);
    }
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

// Whether a product of `tiles` tiles of this kernel has its K shared out
// instead (launch_few): where more than half of the SM pairs would idle and K
// is long beside the tiles.  Measured (us, this kernel / shared out; tiles,
// K blocks): 16, 86 29.0 / 16.8; 16, 43 21.3 / 14.9; 4, 32 13.8 / 8.1; 16, 24
// 11.6 / 10.5; 32, 64 23.0 / 21.2; 16, 16 9.4 / 9.7; 24, 16 9.5 / 12.2; 32, 32
// 14.0 / 14.9.
bool share_k(int64_t tiles, int64_t K)
{
    const int64_t kb = (K + kBK - 1) / kBK;
    return 2 * tiles <= kB200Sms / 2 && kb >= 20 && 2 * kb >= 3 * tiles;
}

// Whether the few-token kernel serves M rows with `tiles` column tiles of this
// kernel.  Up to 64 rows always: this kernel would multiply mostly zeros.
// Beyond, while the tiles leave pairs of SMs idle that shares of K use: all
// of them at 65-128 rows, half at 129-256 (K 4096, us, few tokens / this
// kernel: 64 tiles, M 128 41.8 / 43.9 and 256 50.1 / 43.8; 32 tiles, M 256
// 32.9 / 36.9; 128 tiles, M 64 63.5 / 69.6 and 128 72.7 / 69.6).
bool few_tokens(int64_t M, int64_t tiles)
{
    constexpr int64_t pairs = kB200Sms / 2;
    return M <= 64 || (M <= 128 && tiles <= pairs) || (M <= kFewTokens && 2 * tiles <= pairs);
}

cudaError_t launch_gated(const GatedLaunch &a)
{
    const int64_t rows = (a.M + kBM - 1) / kBM;
    // the backward's heavier epilogue is not hidden there: one tile of tokens
    // ([100 x 4096 x 2048] 21.6 -> 9.4 us, but [512 x 1024 x 2048] 19.6 -> 21.4)
    if (a.mode == 1)
        return a.M <= kFewTokens && share_k((a.N + kAcc - 1) / kAcc, a.K) ? launch_few(a, kFewBwd) : by_act<kBwd>(a);
    const int64_t cols = (a.N + kHalf - 1) / kHalf;
    return few_tokens(a.M, cols) || share_k(rows * cols, a.K) ? launch_few(a, kFewGated) : by_act<kFwd>(a);
}

cudaError_t launch_matmul(const MatmulPlain &p)
{
    GatedLaunch a{};
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.x = p.a;
    a.w0 = p.b;
    a.z = p.c;
    a.stream = p.stream;
    const int64_t cols = (a.N + kAcc - 1) / kAcc, tiles = (a.M + kBM - 1) / kBM * cols;
    const FewKind kind = p.trans_a ? kFewTN : p.trans_b ? kFewNT : kFewNN;
    if ((!p.trans_a && few_tokens(a.M, cols)) || share_k(tiles, a.K)) return launch_few(a, kind);
    if (p.trans_a) return launch_one<ReLU, kPlainTN>(a);
    return p.trans_b ? launch_one<ReLU, kPlainNT>(a) : launch_one<ReLU, kPlainNN>(a);
}

}  // namespace mea
