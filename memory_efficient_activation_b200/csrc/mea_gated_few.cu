// mea_gated_few.cu -- matrix products of few output tiles: the gated
// projections, their backward and plain products in three layouts.
//
// With few rows of X the work is to stream the weights once: 4 N K bytes for
// both projections against 4 M N K operations.  The tensor-core tile is
// therefore turned around: 128 rows of weight are the instruction's M and the
// tokens, rounded up to 16 (at most 256 a tile), its N, so one token wastes 15
// columns of a small operand instead of 255 rows of a large one.
//
// A CTA owns 64 hidden units (64 rows of Wg above the same 64 of Wu; 128 rows
// of W in the plain product) of one tile of tokens, and one of KS shares of
// K; the KS CTAs of a tile form a cluster.  KS is chosen so that the grid
// fills the GPU with about two CTAs per SM: with one CTA per tile, 8192 hidden
// units are 128 CTAs for 148 SMs and 4096 only 64.  Every CTA accumulates in
// tensor memory, leaves its fp32 partial tile in its own shared memory, and
// after a cluster barrier the CTAs share the output tokens out among
// themselves, each adding the KS partials in rank order through distributed
// shared memory: no workspace, one launch, the same bits every time.
//
// In the plain products either operand may be stored with K outermost (its
// tile is then M- or N-major in shared memory): no transposed copies.
//
// Per CTA: warp 0 loads (TMA, 128-byte swizzle) into a ring of 64-wide K
// blocks, warp 1 issues the MMAs, warps 2-5 read the accumulator; all of them
// form the outputs.  Every wait is bounded; one that expires is recorded.
//
// Bound by memory for few tokens: [1 x 4096] to 2 x 8192, 134 MB of weights,
// 25 us, 5.4 TB/s; [37 x 4096] to 2 x 4096, 67 MB, 16 us, of which about 5
// are the launch, the first loads and the join.
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

__device__ unsigned int g_few_error = 0;

namespace {

constexpr int kRowsW = 128;                                  // weight rows of a tile
constexpr int kBK = 64;
constexpr int kThreadsF = 192;
constexpr int kFewSmemMax = 220 * 1024;
constexpr uint32_t kBytesW = kRowsW * kBK * 2;               // 16 KB of weight per stage

__device__ __forceinline__ void record_error() { atomicExch(&g_few_error, 1u); }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void umma_bf16(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 consecutive fp32 columns of this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16])
{
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

struct FewArgs {
    CUtensorMap x, w0, w1;
    int M, N, K;
    int mt;                  // tokens of a tile, a multiple of 16 (64 where A is [K x M])
    int stages;
    uint32_t tmem_cols;
    float param;
    const uint16_t *zin;     // backward: the stored [M x 2N]
    uint16_t *z;             // gated: [M x 2N] or NULL; backward: dz; plain: C
    uint16_t *h;             // gated, backward: [M x N] or NULL
};

// A == void: the plain product; with WN (and an activation) the gated
// backward, otherwise its forward.  KS: CTAs of a cluster, shares of K.  WN:
// the weight is stored [K x N]; XM: X is stored [K x M].
template <class A, int KS, bool WN, bool XM>
__global__ void __launch_bounds__(kThreadsF)
few_kernel(const __grid_constant__ FewArgs a)
{
    constexpr bool kBwd = !std::is_same<A, void>::value && WN;
    constexpr bool kGated = !std::is_same<A, void>::value && !WN;
    constexpr int kCols = kGated ? kRowsW / 2 : kRowsW;      // output columns of a tile
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[8], empty[8], acc_full;
    __shared__ uint32_t tmem_slot;
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    // neighbouring clusters take the same columns for the next tokens, so that
    // a weight tile is read from memory once
    const int tile = (int)(blockIdx.x / KS), tok_tiles = (a.M + a.mt - 1) / a.mt;
    const int n0 = tile / tok_tiles * kCols, m0 = tile % tok_tiles * a.mt;
    const int kb_all = (a.K + kBK - 1) / kBK;
    const int kb0 = (int)((int64_t)kb_all * rank / KS), kbs = (int)((int64_t)kb_all * (rank + 1) / KS) - kb0;
    const uint32_t stage_bytes = kBytesW + (uint32_t)a.mt * (kBK * 2);

    if (threadIdx.x == 32) {
        prefetch_map(&a.x);
        prefetch_map(&a.w0);
        if (kGated) prefetch_map(&a.w1);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_addr(full + s), 1);
            mbar_init(smem_addr(empty + s), 1);
        }
        mbar_init(smem_addr(&acc_full), 1);
        mbar_init_fence();
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(a.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    // the partial tile: token by token, 128 weight rows each
    float *part = reinterpret_cast<float *>(smem);
    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int it = 0;
            for (; it < kbs && ok; ++it) {
                const int s = it % a.stages, round = it / a.stages;
                if (round > 0 && !mbar_wait(smem_addr(empty + s), (round & 1) ^ 1)) {
                    record_error();
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_addr(full + s), sa = sbase + s * stage_bytes;
                const int k = (kb0 + it) * kBK;
                mbar_arrive_expect_tx(bar, stage_bytes);
                if constexpr (WN) {
                    tma_load_2d(sa, &a.w0, n0, k, bar);
                    tma_load_2d(sa + kBytesW / 2, &a.w0, n0 + 64, k, bar);
                } else {
                    tma_load_2d(sa, &a.w0, k, n0, bar);
                    tma_load_2d(sa + kBytesW / 2, kGated ? &a.w1 : &a.w0, k, kGated ? n0 : n0 + 64, bar);
                }
                if constexpr (XM)
                    for (int i = 0; i < a.mt / 64; ++i) tma_load_2d(sa + kBytesW + i * 8192, &a.x, m0 + 64 * i, k, bar);
                else
                    tma_load_2d(sa + kBytesW, &a.x, k, m0, bar);
            }
            for (int j = it > a.stages ? it - a.stages : 0; j < it; ++j)
                if (!mbar_wait(smem_addr(empty + j % a.stages), (j / a.stages) & 1)) record_error();
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // fp32 accumulator, A and B bf16, N = mt, M = 128, each K-major or not
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (WN ? 1u << 15 : 0u) | (XM ? 1u << 16 : 0u) |
                                   ((uint32_t)(a.mt >> 3) << 17) | ((uint32_t)(kRowsW >> 4) << 24);
            bool ok = true;
            for (int it = 0; it < kbs && ok; ++it) {
                const int s = it % a.stages;
                if (!mbar_wait(smem_addr(full + s), (it / a.stages) & 1)) {
                    record_error();
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = sbase + s * stage_bytes;
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    umma_bf16(tmem, WN ? sdesc_mn(sa + k * 2048) : sdesc_sw128(sa + k * 32),
                              XM ? sdesc_mn(sa + kBytesW + k * 2048) : sdesc_sw128(sa + kBytesW + k * 32), idesc,
                              (it | k) != 0);
                umma_commit(smem_addr(empty + s));
            }
            if (ok) umma_commit(smem_addr(&acc_full));
        }
        __syncwarp();
    } else {
        const int q = warp & 3, row = q * 32 + lane;
        if (!mbar_wait(smem_addr(&acc_full), 0)) {
            record_error();
        } else {
            tc_fence_after();
            // every MMA has read its operands: the ring becomes the partial tile
            for (int c = 0; c < a.mt; c += 16) {
                uint32_t v[16];
                tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * kRowsW + row] = __uint_as_float(v[j]);
            }
            tc_fence_before();
        }
    }
    pdl_trigger();
    __syncthreads();
    if (KS > 1) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.tmem_cols) : "memory");
    }

    // outputs: tokens rank, rank + KS, ...; four neighbouring columns per
    // thread, whose partials of all ranks are read before they are added
    auto total = [&](int row, int m) {
        const uint32_t at = smem_addr(part + m * kRowsW + row);
        float4 v[KS];
#pragma unroll
        for (int r = 0; r < KS; ++r)
            v[r] = KS == 1 ? *reinterpret_cast<const float4 *>(part + m * kRowsW + row) : ld_cluster(cluster_addr(at, r));
#pragma unroll
        for (int r = 1; r < KS; ++r) {
            v[0].x += v[r].x;
            v[0].y += v[r].y;
            v[0].z += v[r].z;
            v[0].w += v[r].w;
        }
        return v[0];
    };
    auto put = [](uint16_t *p, float4 v) {         // N is a multiple of 8: four columns are there or none
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    };
    constexpr int kQuads = kCols / 4;
    const int toks = a.M - m0 < a.mt ? a.M - m0 : a.mt;    // of the tile; mine: of this rank
    const int mine = (toks - (int)rank + KS - 1) / KS;
    for (int i = threadIdx.x; i < mine * kQuads; i += kThreadsF) {
        const int t = (int)rank + i / kQuads * KS, c = i % kQuads * 4, n = n0 + c;
        const int64_t m = m0 + t;
        if (n >= a.N) continue;
        if constexpr (kGated) {
            const float4 g = total(c, t), u = total(kCols + c, t);
            if (a.z) {
                uint16_t *z = a.z + m * 2 * a.N + n;
                put(z, g);
                put(z + a.N, u);
            }
            if (a.h) {
                const Coef k = A::coef(a.param);
                bool tail = false;
                float4 f = make_float4(A::template f<false>(g.x, k, tail), A::template f<false>(g.y, k, tail),
                                       A::template f<false>(g.z, k, tail), A::template f<false>(g.w, k, tail));
                if (tail) {
                    if (A::is_tail(g.x, k)) f.x = A::template f_tail<false>(g.x, k);
                    if (A::is_tail(g.y, k)) f.y = A::template f_tail<false>(g.y, k);
                    if (A::is_tail(g.z, k)) f.z = A::template f_tail<false>(g.z, k);
                    if (A::is_tail(g.w, k)) f.w = A::template f_tail<false>(g.w, k);
                }
                put(a.h + m * a.N + n, make_float4(f.x * u.x, f.y * u.y, f.z * u.z, f.w * u.w));
            }
        } else if constexpr (kBwd) {
            const float4 d = total(c, t);
            const uint16_t *zi = a.zin + m * 2 * a.N + n;
            const uint2 gw = *reinterpret_cast<const uint2 *>(zi), uw = *reinterpret_cast<const uint2 *>(zi + a.N);
            const float dv[4] = {d.x, d.y, d.z, d.w};
            const float gv[4] = {__uint_as_float(gw.x << 16), __uint_as_float(gw.x & 0xffff0000u),
                                 __uint_as_float(gw.y << 16), __uint_as_float(gw.y & 0xffff0000u)};
            const float uv[4] = {__uint_as_float(uw.x << 16), __uint_as_float(uw.x & 0xffff0000u),
                                 __uint_as_float(uw.y << 16), __uint_as_float(uw.y & 0xffff0000u)};
            const Coef k = A::coef(a.param);
            float dg[4], du[4], hv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bool tail = false;
                float v = A::template f<false>(gv[e], k, tail);
                if (tail && A::is_tail(gv[e], k)) v = A::template f_tail<false>(gv[e], k);
                hv[e] = v * uv[e];
                du[e] = v * dv[e];
                tail = false;
                dg[e] = A::template df<false>(gv[e], dv[e] * uv[e], k, tail);
                if (tail && A::template is_tail_bwd<false>(gv[e], k))
                    dg[e] = A::template df_tail<false>(gv[e], dv[e] * uv[e], k);
            }
            uint16_t *z = a.z + m * 2 * a.N + n;
            put(z, make_float4(dg[0], dg[1], dg[2], dg[3]));
            put(z + a.N, make_float4(du[0], du[1], du[2], du[3]));
            if (a.h) put(a.h + m * a.N + n, make_float4(hv[0], hv[1], hv[2], hv[3]));
        } else {
            put(a.z + m * a.N + n, total(c, t));
        }
    }
    if (KS > 1) cluster_sync();                    // no CTA leaves while its partials may be read
}

// ------------------------------------------------------------ host side

template <class A, int KS, bool WN, bool XM>
cudaError_t launch_ks(const FewArgs &a, int64_t tiles, size_t smem, cudaStream_t stream)
{
    auto kernel = few_kernel<A, KS, WN, XM>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * KS));
    cfg.blockDim = dim3(kThreadsF);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = KS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <class A, bool WN, bool XM>
cudaError_t launch_few_one(const GatedLaunch &g)
{
    constexpr bool kGated = !std::is_same<A, void>::value && !WN;
    FewArgs a;
    a.zin = static_cast<const uint16_t *>(g.zin);
    a.M = (int)g.M;
    a.N = (int)g.N;
    a.K = (int)g.K;
    const int64_t toks = (g.M + kFewTokens - 1) / kFewTokens;
    constexpr int kRound = XM ? 64 : 16;
    a.mt = (int)(((g.M + toks - 1) / toks + kRound - 1) / kRound * kRound);
    a.param = g.param;
    a.z = static_cast<uint16_t *>(g.z);
    a.h = static_cast<uint16_t *>(g.h);
    const bool ok = (XM ? bf16_tile_map(&a.x, g.x, g.K, g.M, kBK) : bf16_tile_map(&a.x, g.x, g.M, g.K, (uint32_t)a.mt)) &&
                    (WN ? bf16_tile_map(&a.w0, g.w0, g.K, g.N, kBK) : bf16_tile_map(&a.w0, g.w0, g.N, g.K, 64));
    if (!ok) return cudaErrorInvalidValue;
    a.w1 = a.w0;
    if (kGated && !bf16_tile_map(&a.w1, g.w1, g.N, g.K, 64)) return cudaErrorInvalidValue;
    // Shares of K: as many as keep the grid within two CTAs per SM, each with
    // at least four K blocks.  Up to 144 tokens a tile three stages fit half an
    // SM's shared memory; beyond, one CTA per SM, and clusters of four at most:
    // eight whole SMs of one GPC are hard to come by ([100 x 4096] x 2048 16.1
    // us as one CTA per SM and eight, 11.0 four, 10.3 two and eight; [200 x
    // 4096] x 2048 20.2 eight, 12.7 four).
    const int cols = kGated ? kRowsW / 2 : kRowsW;
    const int64_t tiles = (g.N + cols - 1) / cols * ((g.M + a.mt - 1) / a.mt), kb = (g.K + kBK - 1) / kBK;
    const uint32_t stage = kBytesW + (uint32_t)a.mt * (kBK * 2);
    const int per_sm = stage <= 34 * 1024 ? 2 : 1;
    int ks = 1;
    while (ks < 4 * per_sm && tiles * ks * 2 <= (int64_t)kB200Sms * per_sm && kb >= ks * 2 * 4) ks *= 2;
    const uint32_t budget = (uint32_t)kFewSmemMax / per_sm - 2048;
    a.stages = (int)(budget / stage) < 8 ? (int)(budget / stage) : 8;
    a.tmem_cols = 32;
    while (a.tmem_cols < (uint32_t)a.mt) a.tmem_cols *= 2;
    const size_t part = (size_t)kRowsW * a.mt * sizeof(float);
    size_t smem = (size_t)a.stages * stage;
    if (smem < part) smem = part;
    smem += 1024;
    // the gated backward and a transposed A come here for a share of K only
    // (at most 74 tiles of this width, 20 K blocks or more)
    constexpr bool kShared = (!std::is_same<A, void>::value && WN) || XM;
    switch (ks) {
    case 1:
        if constexpr (!kShared) return launch_ks<A, 1, WN, XM>(a, tiles, smem, g.stream);
        return cudaErrorInvalidValue;
    case 2: return launch_ks<A, 2, WN, XM>(a, tiles, smem, g.stream);
    case 4: return launch_ks<A, 4, WN, XM>(a, tiles, smem, g.stream);
    }
    return launch_ks<A, 8, WN, XM>(a, tiles, smem, g.stream);
}

template <bool WN>
cudaError_t few_by_act(const GatedLaunch &g)
{
    switch (g.act) {
    case 0: return launch_few_one<ReLU, WN, false>(g);
    case 1: return launch_few_one<LeakyReLU, WN, false>(g);
    case 2: return launch_few_one<Sigmoid, WN, false>(g);
    case 3: return launch_few_one<Tanh, WN, false>(g);
    case 4: return launch_few_one<GeluErf, WN, false>(g);
    case 5: return launch_few_one<GeluTanh, WN, false>(g);
    case 6: return launch_few_one<SwishT<WN>, WN, false>(g);     // f alone has no zero of f' to guard
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t few_error_word(int clear, unsigned int *word)
{
    cudaError_t e = cudaMemcpyFromSymbol(word, g_few_error, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_few_error, &zero, sizeof(unsigned int));
    }
    return e;
}

cudaError_t launch_few(const GatedLaunch &g, FewKind kind)
{
    switch (kind) {
    case kFewNT: return launch_few_one<void, false, false>(g);
    case kFewNN: return launch_few_one<void, true, false>(g);
    case kFewTN: return launch_few_one<void, true, true>(g);
    case kFewGated: break;
    case kFewBwd: return few_by_act<true>(g);
    }
    return few_by_act<false>(g);
}

}  // namespace mea
