// mea_norm.cu -- normalisation of rows (the last axis): layer norm and rms
// norm, forward and backward.
//
//   forward    mean = sum x / C (0 for rms), invstd = 1 / sqrt(var + eps),
//              var = sum (x - mean)^2 / C, xhat = (x - mean) invstd,
//              y = gamma xhat + beta
//   backward   a = dy gamma, m1 = sum a / C (0 for rms), m2 = sum a xhat / C,
//              dx = invstd (a - m1 - xhat m2),
//              dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy
//
// Both are bound by memory (8 to 14 operations per element), so each tensor is
// read once.  The variance is a second pass over the row on chip (sum of (x -
// mean)^2; in the forward's ring over each warp's part of it from that part's
// mean, the parts merged), not a difference of two large sums.  Row sums are fp32, short
// sequences in a thread and then a tree; column sums take at most 1024 rows in
// fp32 and add those in fp64.  Every kernel's results are rounded once.
//
// Forward, by shape:
//   many rows of 33 to 512 vectors    a warp to a row, in registers
//   other large tensors               blocks over shared-memory rings
//   small tensors (below 4 MB)        a row spread over more threads
//   rows no block's registers hold    three passes over the row
// Backward:
//   rows that 512 threads hold        one pass over x and dy for dx and the
//                                     column sums, over shared-memory rings
//   longer rows, unaligned tensors    column sums, then dx
//
// Measured back to back, 16384 x 4096 bf16 with fp32 parameters: forward 48 us
// (5.6 TB/s), backward with the join of dgamma and dbeta 80 (5.0 TB/s), or 74
// replayed from a graph on the same buffers.
// What bounds the backward is latency at 16 warps per SM: 170 instructions a
// warp and 256 elements issue in 57 percent of the cycles; two blocks of 64
// registers (and two rows between barriers) were slower.
#include <cuda_runtime.h>

#include <cstdint>

#include "mea_device.cuh"
#include "mea_internal.h"
#include "mea_math.cuh"
#include "mea_norm_api.h"
#include "mea_pipe.cuh"
#include "mea_stream.cuh"

namespace mea {

__device__ unsigned int g_norm_error = 0;   // a bounded barrier wait expired

namespace {

constexpr int kNormThreads = 256;      // threads of a block (more where one row needs more)
constexpr int kNormMaxThreads = 1024;
constexpr int kSlabRows = 1024;        // most rows whose terms one fp32 column sum takes
constexpr int kSlabs = kB200Sms;       // column-sum slabs of a large tensor
// Size of x from which the forward streams through a ring (us, one row per
// group of threads / ring: 1001 bf16 channels, 2 MB 3.9 / 6.8, 4 MB 8.9 / 8.8,
// 8 MB 22.0 / 12.0; 144 bf16 2 MB 2.6 / 3.1, 8 MB 8.5 / 8.1).
constexpr int64_t kRingBytes = 4 << 20;
constexpr int kColX = 32, kColY = 8;   // threads of a column-sum block: columns x rows

// Column-sum slabs, from the row count and the rows a block takes at a time
// only, so the order of the sums does not depend on the device: one block per
// SM, at least one round of rows each, at most kSlabRows rows.
inline int64_t norm_slabs(int64_t rows, int at_a_time)
{
    int64_t s = (rows + at_a_time - 1) / at_a_time;
    if (s > kSlabs) s = kSlabs;
    const int64_t m = (rows + kSlabRows - 1) / kSlabRows;
    if (s < m) s = m;
    return s < 1 ? 1 : s;
}

// VL parameters from item i (elements i VL ..), or `fill` where p is NULL.
template <typename TP, int VL>
__device__ __forceinline__ void load_params(const void *p, int64_t i, float fill, float (&f)[VL])
{
    if (!p) {
#pragma unroll
        for (int j = 0; j < VL; ++j) f[j] = fill;
    } else if constexpr (VL == 1) {
        f[0] = Store<TP>::load1(p, i);
    } else {
        constexpr int PV = Store<TP>::V;
        constexpr int n = VL < PV ? VL : PV;   // elements taken from each 16-byte vector (or half of one)
        if constexpr (VL < PV) {
            // four bf16 parameters beside four fp32 elements: 8 bytes
            const uint2 w = __ldg(static_cast<const uint2 *>(p) + i);
            f[0] = __uint_as_float(w.x << 16);
            f[1] = __uint_as_float(w.x & 0xffff0000u);
            f[2] = __uint_as_float(w.y << 16);
            f[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
#pragma unroll
            for (int q = 0; q < VL / n; ++q) {
                const uint4 w = __ldg(static_cast<const uint4 *>(p) + i * (VL / n) + q);
                float t[PV];
                Store<TP>::unpack(w, t);
#pragma unroll
                for (int j = 0; j < n; ++j) f[q * n + j] = t[j];
            }
        }
    }
}

// Sum over the 2^lg (at most 32) neighbouring threads of a warp that share a
// row, in each of them.
__device__ __forceinline__ float lanes_sum(float v, int lg)
{
    if (lg >= 5) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    } else {
        for (int b = 0; b < lg; ++b) v += __shfl_xor_sync(0xffffffffu, v, 1 << b);
    }
    return v;
}

// Sum over the group of 2^lg threads that owns a row, in every thread of the
// group.  Groups of more than a warp exchange through red (one float per
// warp), between two barriers that every thread of the block takes.
__device__ __forceinline__ float group_sum(float v, int lg, float *red)
{
    v = lanes_sum(v, lg);
    if (lg > 5) {
        const int warp = threadIdx.x >> 5, wpg = 1 << (lg - 5), first = warp & ~(wpg - 1);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < wpg; ++w) v += red[first + w];
    }
    return v;
}

// Arithmetic on the elements of an item, two at a time in packed .f32x2
// instructions (the one-pass kernels are near the issue limit without them).
template <int VL>
__device__ __forceinline__ void v_center(float (&x)[VL], float m, float s)   // (x - m) s
{
    if constexpr (VL == 1) {
        x[0] = (x[0] - m) * s;
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2) upk(mul2(add2(pk(x[e], x[e + 1]), sp2(-m)), sp2(s)), x[e], x[e + 1]);
    }
}
template <int VL>
__device__ __forceinline__ void v_shift(float (&x)[VL], float m)   // x - m
{
    if constexpr (VL == 1) {
        x[0] -= m;
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2) upk(add2(pk(x[e], x[e + 1]), sp2(-m)), x[e], x[e + 1]);
    }
}
template <int VL>
__device__ __forceinline__ void v_mul(const float (&a)[VL], const float (&b)[VL], float (&o)[VL])
{
    if constexpr (VL == 1) {
        o[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2) upk(mul2(pk(a[e], a[e + 1]), pk(b[e], b[e + 1])), o[e], o[e + 1]);
    }
}
template <int VL>
__device__ __forceinline__ void v_fma(const float (&a)[VL], const float (&b)[VL], float (&o)[VL])   // o += a b
{
    if constexpr (VL == 1) {
        o[0] = fmaf(a[0], b[0], o[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2)
            upk(fma2(pk(a[e], a[e + 1]), pk(b[e], b[e + 1]), pk(o[e], o[e + 1])), o[e], o[e + 1]);
    }
}
template <int VL>
__device__ __forceinline__ void v_add(const float (&a)[VL], float (&o)[VL])   // o += a
{
    if constexpr (VL == 1) {
        o[0] += a[0];
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2) upk(add2(pk(a[e], a[e + 1]), pk(o[e], o[e + 1])), o[e], o[e + 1]);
    }
}
// Two partial sums of the elements, and of the products.
template <int VL>
__device__ __forceinline__ void v_sum(const float (&a)[VL], float (&s)[2])
{
    if constexpr (VL == 1) {
        s[0] += a[0];
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2) upk(add2(pk(a[e], a[e + 1]), pk(s[0], s[1])), s[0], s[1]);
    }
}
template <int VL>
__device__ __forceinline__ void v_dot(const float (&a)[VL], const float (&b)[VL], float (&s)[2])
{
    if constexpr (VL == 1) {
        s[0] = fmaf(a[0], b[0], s[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2)
            upk(fma2(pk(a[e], a[e + 1]), pk(b[e], b[e + 1]), pk(s[0], s[1])), s[0], s[1]);
    }
}
// p a + (h b + c), over p
template <int VL>
__device__ __forceinline__ void v_dx(float (&p)[VL], const float (&h)[VL], float a, float b, float c)
{
    if constexpr (VL == 1) {
        p[0] = fmaf(p[0], a, fmaf(h[0], b, c));
    } else {
#pragma unroll
        for (int e = 0; e < VL; e += 2)
            upk(fma2(pk(p[e], p[e + 1]), sp2(a), fma2(pk(h[e], h[e + 1]), sp2(b), sp2(c))), p[e], p[e + 1]);
    }
}

// ------------------------------------------------------------- row rings
//
// The one-pass kernels: a block takes a run of consecutive rows through a ring
// of stages in shared memory that 1-D bulk copies fill (rows are contiguous:
// one copy per tensor and stage), far enough ahead that a row reduction's
// barrier does not show.  G threads own a row, NV items of VL elements each,
// and S = threads / G rows lie side by side.  A thread keeps the same columns
// of every row it sees, so gamma and beta (and the backward's column sums)
// stay in registers.
//
// Copies start and end on 16-byte boundaries: a stage whose rows do not is
// copied from the boundary before it (its elements then lie `skew` further
// on) to the one after, except at the very end of the tensor, whose last few
// elements are read directly.
//
// G is a power of two up to a warp, or a number of whole warps.
struct RingGeo {
    int G, S, nv;            // threads to a row, rows at a time, items per thread
};

// The copy of a stage and a thread's view of it.
template <typename T, int VL>
struct RingView {
    static constexpr int q = 16 / Store<T>::kBytes;
    // Elements [a, b) of a tensor of `end` elements into the stage at dst:
    // the bytes of the bulk copy, which starts on the boundary at or before a.
    // One thread calls this; the copy completes on `bar`, the few elements
    // that a copy to the boundary after the tensor's end would overrun are
    // stored here (a barrier of the block comes between that and their use).
    static __device__ __forceinline__ uint32_t bytes(int64_t a, int64_t b, int64_t end)
    {
        const int64_t up = (b + q - 1) & ~(int64_t)(q - 1);
        return (uint32_t)(((up <= end ? up : b & ~(int64_t)(q - 1)) - (a & ~(int64_t)(q - 1))) * Store<T>::kBytes);
    }
    static __device__ __forceinline__ void copy(unsigned char *dst, const void *p, int64_t a, int64_t b, uint32_t n,
                                                uint32_t bar)
    {
        const int64_t first = a & ~(int64_t)(q - 1);
        if (n) bulk_load(smem_addr(dst), static_cast<const unsigned char *>(p) + first * Store<T>::kBytes, n, bar);
        if constexpr (VL == 1)
            for (int64_t i = first + n / Store<T>::kBytes; i < b; ++i)
                Store<T>::store1(dst, i - first, Store<T>::load1_rw(p, i));
    }
    uint32_t at;             // this thread's item 0: elements from the rows' start in the stage
    uint32_t skew, turn;     // VL 1: elements before the rows' start, and their change per step
    __device__ __forceinline__ RingView(int64_t r0, int64_t C, int per, int slot, int g)
    {
        at = (uint32_t)(slot * C) + g * VL;
        skew = VL == 1 ? (uint32_t)((r0 * C) & (q - 1)) : 0u;
        turn = VL == 1 ? (uint32_t)((per * C) & (q - 1)) : 0u;
    }
    __device__ __forceinline__ void next()
    {
        if constexpr (VL == 1) skew = (skew + turn) & (q - 1);
    }
    // The i-th item after item 0 in the row that starts `off` elements after
    // this thread's first.
    __device__ __forceinline__ void load(const unsigned char *stage, int i, int off, float (&f)[VL]) const
    {
        if constexpr (VL == 1)
            f[0] = Store<T>::load1_rw(stage, skew + at + off + i);
        else
            Store<T>::unpack(*reinterpret_cast<const uint4 *>(stage + (at + off + i * VL) * Store<T>::kBytes), f);
    }
};

__device__ __forceinline__ int lane_bits(int G) { return G >= 32 ? 5 : __ffs(G) - 1; }

// ---------------------------------------------------------------- forward

template <typename T, typename TP, bool RMS, int VL, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS)
norm_fwd_kernel(const void *__restrict__ x, const void *__restrict__ gamma, const void *__restrict__ beta, float eps,
                void *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ invstd_out, int64_t rows,
                int64_t C, int lg)
{
    using It = Item<T, VL>;
    __shared__ float red[32];
    const int g = threadIdx.x & ((1 << lg) - 1), G = 1 << lg;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> lg) + (threadIdx.x >> lg);
    const bool live = row < rows;
    const int items = (int)(C / VL);
    const int64_t base = row * items;
    const float rc = 1.f / (float)C;
    pdl_wait();
    typename It::Raw r[NV];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) r[j] = It::load(x, base + g + j * G);
    float mean = 0.f;
    if constexpr (!RMS) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && g + j * G < items) {
                float f[VL];
                It::unpack(r[j], f);
                s += tree_sum(f);
            }
        mean = group_sum(s, lg, red) * rc;
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) {
            float f[VL];
            It::unpack(r[j], f);
#pragma unroll
            for (int e = 0; e < VL; ++e) {
                f[e] -= mean;
                f[e] *= f[e];
            }
            q += tree_sum(f);
        }
    const float invstd = rsqrtf(fmaf(group_sum(q, lg, red), rc, eps));
    pdl_trigger();
    if (!live) return;
    if (g == 0) {
        if (!RMS && mean_out) mean_out[row] = mean;
        if (invstd_out) invstd_out[row] = invstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (g + j * G < items) {
            float f[VL], w[VL], b[VL];
            It::unpack(r[j], f);
            load_params<TP, VL>(gamma, g + j * G, 1.f, w);
            load_params<TP, VL>(beta, g + j * G, 0.f, b);
#pragma unroll
            for (int e = 0; e < VL; ++e) f[e] = fmaf((f[e] - mean) * invstd, w[e], b[e]);
            It::store(y, base + g + j * G, f);
        }
}

constexpr int kRingThreads = 512;

// Sums over the row's G threads of N values (sums of R rows), N a power of
// two: returns them in v, in every thread of the group.  Groups within a warp
// shuffle each value.  Larger ones halve the values at every step of the
// butterfly until each lane holds part of one, exchange through red (N floats
// per warp) and the block's barrier, and spread the totals by shuffles.
// Every thread of the block takes part, once per barrier in turn.
template <int N>
__device__ __forceinline__ void reduce_rows(float (&v)[N], int G, int w0, float (*red)[N][16])
{
    const int lane = threadIdx.x & 31;
    if (G < 32) {
        const int lb = lane_bits(G);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lanes_sum(v[i], lb);
        __syncthreads();
        return;
    }
    constexpr int L = N == 8 ? 3 : N == 4 ? 2 : N == 2 ? 1 : 0;
    static_assert(N == 1 << L, "a power of two of values");
#pragma unroll
    for (int b = 0; b < 5; ++b) {
        const int off = 16 >> b;
        if (b < L) {
            const bool hi = lane & off;
#pragma unroll
            for (int i = 0; i < (N >> (b + 1)); ++i) {
                const float keep = hi ? v[i + (N >> (b + 1))] : v[i], give = hi ? v[i] : v[i + (N >> (b + 1))];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        }
    }
    // lane: value lane >> (5 - L)
    constexpr int kPart = 32 >> L;                 // lanes of one value
    const int mine = lane / kPart, part = lane % kPart, wpg = G >> 5;
    if (part == 0) (*red)[mine][threadIdx.x >> 5] = v[0];
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 16; k += kPart < 16 ? kPart : 16)
        if (part + k < wpg) t += (*red)[mine][w0 + part + k];
#pragma unroll
    for (int off = kPart / 2; off >= 1; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t, i * kPart);
}

// Forward of a run of rows, 16 elements of a row per thread where they fit.
// Layer norm's variance needs the mean first; to take one barrier instead of
// two, every warp forms the sum of its own elements and their squared
// distances from the warp's own mean, and the row's warps are merged exactly
// (Chan, Golub and LeVeque, "Updating formulae and a pairwise algorithm for
// computing sample variances", 1979):
//   M2 = sum M2_w + sum n_w (mean_w - mean)^2.
// Blocks of 256 threads, three to an SM (two for long rows): one row at a time
// and more warps measured better here than the backward's several rows
// between barriers (16384 x 4096 bf16: 62 against 79 us).
constexpr int kFwdThreads = 256;
template <typename T, int VL, int NV>
struct FwdRing {
    static constexpr bool kKeep = VL * NV <= 16;   // gamma and beta in registers
    static constexpr int kBlocks = kKeep ? 3 : 2;  // per SM
    static constexpr uint32_t bytes = (uint32_t)kFwdThreads * NV * VL * Store<T>::kBytes + 32;
    static constexpr int kFit = (int)((kKeep ? 72u : 108u) * 1024 / bytes);
    static constexpr int stages = kFit < 8 ? kFit : 8;
    static constexpr size_t smem = (size_t)stages * bytes;
    static_assert(stages >= (VL == 1 ? 2 : 1), "single elements: a barrier between filling a stage and using it");
};

template <typename T, typename TP, bool RMS, int VL, int NV>
__global__ void __launch_bounds__(kFwdThreads, FwdRing<T, VL, NV>::kBlocks)
norm_fwd_ring_kernel(const void *__restrict__ x, const void *__restrict__ gamma, const void *__restrict__ beta,
                     float eps, void *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ invstd_out,
                     int64_t rows, int64_t C, int G, int S, int64_t per_block)
{
    using F = FwdRing<T, VL, NV>;
    using V = RingView<T, VL>;
    constexpr int kRing = F::stages, eb = Store<T>::kBytes;
    constexpr uint32_t kBytes = F::bytes;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kRing];
    __shared__ float red[2][2][8];
    const int tid = threadIdx.x, slot = tid / G, g = tid - slot * G, lb = lane_bits(G), wpg = G >> 5;
    const int w0 = slot * wpg, lane = tid & 31;
    const int items = (int)(C / VL);
    const int64_t r0 = (int64_t)blockIdx.x * per_block, r1 = r0 + per_block < rows ? r0 + per_block : rows;
    const int steps = r1 > r0 ? (int)((r1 - r0 + S - 1) / S) : 0;
    const float rc = 1.f / (float)C;
    if (tid == 0) {
        for (int s = 0; s < kRing; ++s) mbar_init(smem_addr(full + s), 1);
        mbar_init_fence();
    }
    __syncthreads();
    pdl_wait();
    auto fill = [&](int s, int st) {
        const int64_t a = r0 + (int64_t)s * S, b = a + S < r1 ? a + S : r1;
        const uint32_t bar = smem_addr(full + st), n = V::bytes(a * C, b * C, rows * C);
        mbar_arrive_expect_tx(bar, n);
        V::copy(ring + st * kBytes, x, a * C, b * C, n, bar);
    };
    if (tid == 0)
        for (int s = 0; s < kRing && s < steps; ++s) fill(s, s);
    if constexpr (VL == 1) __syncthreads();

    float wk[F::kKeep ? NV : 1][VL], bk[F::kKeep ? NV : 1][VL];
    int mine = 0;                                  // this thread's elements of a row
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (g + j * G < items) {
            mine += VL;
            if constexpr (F::kKeep) {
                load_params<TP, VL>(gamma, g + j * G, 1.f, wk[j]);
                load_params<TP, VL>(beta, g + j * G, 0.f, bk[j]);
            }
        }
    // elements of this warp's part of the row (of the whole row for a group
    // within a warp), and of the warp that this lane merges
    const float nw = lanes_sum((float)mine, lb), rnw = nw > 0.f ? 1.f / nw : 0.f;
    float nl = 0.f;
    if (!RMS && G > 32) {
        if (lane == 0) red[0][0][tid >> 5] = nw;
        __syncthreads();
        nl = lane < wpg ? red[0][0][w0 + lane] : 0.f;
        __syncthreads();
    }
    V view(r0, C, S, slot, g);
    int64_t row = r0 + slot;
    const int64_t at0 = (row * C + g * VL) * eb, hop = S * C * eb;
    unsigned char *yp = static_cast<unsigned char *>(y) + at0;
    int st = 0;
    uint32_t turn = 0;
    for (int s = 0; s < steps; ++s, row += S, yp += hop) {
        if (!mbar_wait(smem_addr(full + st), turn)) atomicExch(&g_norm_error, 1u);
        const bool live = row < r1;
        float h[NV][VL];
        float t[2] = {0.f, 0.f};
        if (live) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (g + j * G < items) {
                    view.load(ring + st * kBytes, j * G, 0, h[j]);
                    if (RMS)
                        v_dot(h[j], h[j], t);
                    else
                        v_sum(h[j], t);
                }
        }
        float mean = 0.f, m2;
        if constexpr (RMS) {
            m2 = lanes_sum(t[0] + t[1], lb);
        } else {
            mean = lanes_sum(t[0] + t[1], lb) * rnw;
            t[0] = t[1] = 0.f;
            if (live) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (g + j * G < items) {
                        float c[VL];
#pragma unroll
                        for (int e = 0; e < VL; ++e) c[e] = h[j][e];
                        v_shift(c, mean);
                        v_dot(c, c, t);
                    }
            }
            m2 = lanes_sum(t[0] + t[1], lb);
        }
        if (G > 32 && lane == 0) {
            red[s & 1][0][tid >> 5] = mean;
            red[s & 1][1][tid >> 5] = m2;
        }
        __syncthreads();                           // the rows' sums, and every thread has left the stage
        if (tid == 0 && s + kRing < steps) fill(s + kRing, st);
        if (++st == kRing) {
            st = 0;
            turn ^= 1;
        }
        view.next();
        if (G > 32) {
            const float qw = lane < wpg ? red[s & 1][1][w0 + lane] : 0.f;
            float v = qw;
            if constexpr (!RMS) {
                const float mw = lane < wpg ? red[s & 1][0][w0 + lane] : 0.f;
                float u = mw * nl;
#pragma unroll
                for (int off = 4; off >= 1; off >>= 1) u += __shfl_xor_sync(0xffffffffu, u, off);
                mean = __shfl_sync(0xffffffffu, u, 0) * rc;
                // a lane without a warp adds nothing: its own 0 - mean squared
                // may overflow, and infinity times nl = 0 is no zero
                const float d = nl > 0.f ? mw - mean : 0.f;
                v = fmaf(d * d, nl, qw);
            }
#pragma unroll
            for (int off = 4; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            m2 = __shfl_sync(0xffffffffu, v, 0);
        }
        if (!live) continue;
        const float is = rsqrtf(fmaf(m2, rc, eps));
        if (g == 0) {
            if (!RMS && mean_out) mean_out[row] = mean;
            if (invstd_out) invstd_out[row] = is;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (g + j * G < items) {
                float w[VL], b[VL];
                if constexpr (F::kKeep) {
#pragma unroll
                    for (int e = 0; e < VL; ++e) {
                        w[e] = wk[j][e];
                        b[e] = bk[j][e];
                    }
                } else {
                    load_params<TP, VL>(gamma, g + j * G, 1.f, w);
                    load_params<TP, VL>(beta, g + j * G, 0.f, b);
                }
                v_center(h[j], mean, is);
                v_fma(h[j], w, b);
                Item<T, VL>::store(yp, j * G, b);
            }
    }
    pdl_trigger();
}

// Forward with a warp to a row: 8 warps of a block, two blocks per SM, take
// rows in turn.  A warp holds its row in registers (NV vectors a lane, all of
// their loads in flight at once), sums by shuffles alone and meets no barrier;
// gamma and beta wait in shared memory, where reading them costs no latency
// of L1 and no registers.  Half the instructions of the ring's.
constexpr int kWarpThreads = 256;
template <typename T, typename TP, bool RMS, int NV>
__global__ void __launch_bounds__(kWarpThreads, 2)
norm_fwd_warp_kernel(const void *__restrict__ x, const void *__restrict__ gamma, const void *__restrict__ beta,
                     float eps, void *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ invstd_out,
                     int64_t rows, int64_t C)
{
    constexpr int VL = Store<T>::V;
    // 16-byte words of VL parameters; words apart, so that a warp reads each
    // in one piece
    constexpr int kWords = VL * Store<TP>::kBytes >= 16 ? VL * Store<TP>::kBytes / 16 : 1;
    constexpr bool kHalf = VL * Store<TP>::kBytes < 16;      // four bf16 beside four fp32: 8 bytes
    extern __shared__ uint4 par[];
    const int items = (int)(C / VL), lane = threadIdx.x & 31;
    const float rc = 1.f / (float)C;
    pdl_wait();
    uint4 *sg = par, *sb = par + kWords * items;
    for (int i = threadIdx.x; i < items; i += kWarpThreads) {
        float w[VL], b[VL];
        load_params<TP, VL>(gamma, i, 1.f, w);
        load_params<TP, VL>(beta, i, 0.f, b);
        if constexpr (kHalf) {
            sg[i] = make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(b[0], b[1]),
                               pack_bf16x2(b[2], b[3]));
        } else {
            constexpr int PV = Store<TP>::V;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                float t[PV], u[PV];
#pragma unroll
                for (int e = 0; e < PV; ++e) {
                    t[e] = w[k * PV + e];
                    u[e] = b[k * PV + e];
                }
                sg[k * items + i] = Store<TP>::pack(t);
                sb[k * items + i] = Store<TP>::pack(u);
            }
        }
    }
    __syncthreads();
    auto params = [&](int i, float (&w)[VL], float (&b)[VL]) {
        if constexpr (kHalf) {
            float t[8];
            Store<Bf16>::unpack(sg[i], t);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = t[e];
                b[e] = t[4 + e];
            }
        } else {
            constexpr int PV = Store<TP>::V;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                float t[PV], u[PV];
                Store<TP>::unpack(sg[k * items + i], t);
                Store<TP>::unpack(sb[k * items + i], u);
#pragma unroll
                for (int e = 0; e < PV; ++e) {
                    w[k * PV + e] = t[e];
                    b[k * PV + e] = u[e];
                }
            }
        }
    };
    constexpr int kWarps = kWarpThreads / 32;
    for (int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); row < rows; row += (int64_t)gridDim.x * kWarps) {
        const uint4 *xr = static_cast<const uint4 *>(x) + row * items + lane;
        uint4 *yr = static_cast<uint4 *>(y) + row * items + lane;
        uint4 r[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane + 32 * j < items) r[j] = ld_nc_v4(xr + 32 * j);
        float mean = 0.f, t[2] = {0.f, 0.f};
        if constexpr (!RMS) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (lane + 32 * j < items) {
                    float f[VL];
                    Store<T>::unpack(r[j], f);
                    v_sum(f, t);
                }
            mean = lanes_sum(t[0] + t[1], 5) * rc;
            t[0] = t[1] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane + 32 * j < items) {
                float f[VL];
                Store<T>::unpack(r[j], f);
                if (!RMS) v_shift(f, mean);
                v_dot(f, f, t);
            }
        const float is = rsqrtf(fmaf(lanes_sum(t[0] + t[1], 5), rc, eps));
        if (lane == 0) {
            if (!RMS && mean_out) mean_out[row] = mean;
            if (invstd_out) invstd_out[row] = is;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane + 32 * j < items) {
                float f[VL], w[VL], b[VL];
                Store<T>::unpack(r[j], f);
                params(lane + 32 * j, w, b);
                v_center(f, mean, is);
                v_fma(f, w, b);
                st_v4(yr + 32 * j, Store<T>::pack(b));
            }
    }
    pdl_trigger();
}

// Rows too long for the registers of a block: one block per row, which is
// read again for each of the passes.
template <typename T, typename TP, bool RMS>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_fwd_long_kernel(const void *__restrict__ x, const void *__restrict__ gamma, const void *__restrict__ beta,
                     float eps, void *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ invstd_out,
                     int64_t rows, int64_t C)
{
    __shared__ double red[32];
    __shared__ float bc;
    const int64_t row = blockIdx.x, base = row * C;
    pdl_wait();
    float mean = 0.f;
    if constexpr (!RMS) {
        double s = 0.0;
        for (int64_t i = threadIdx.x; i < C; i += blockDim.x) s += Store<T>::load1(x, base + i);
        s = block_sum(s, red);
        if (threadIdx.x == 0) bc = (float)(s / (double)C);
        __syncthreads();
        mean = bc;
        __syncthreads();
    }
    double q = 0.0;
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float d = Store<T>::load1(x, base + i) - mean;
        q += (double)d * d;
    }
    q = block_sum(q, red);
    if (threadIdx.x == 0) bc = rsqrtf((float)(q / (double)C) + eps);
    __syncthreads();
    const float invstd = bc;
    pdl_trigger();
    if (threadIdx.x == 0) {
        if (!RMS && mean_out) mean_out[row] = mean;
        if (invstd_out) invstd_out[row] = invstd;
    }
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float w = gamma ? Store<TP>::load1(gamma, i) : 1.f, b = beta ? Store<TP>::load1(beta, i) : 0.f;
        Store<T>::store1(y, base + i, fmaf((Store<T>::load1(x, base + i) - mean) * invstd, w, b));
    }
}

// --------------------------------------------------------------- backward

// Column sums of one slab of rows: partial[slab][0][c] = sum dy xhat,
// partial[slab][1][c] = sum dy.  A block covers 32 VL columns with 8 rows at
// a time; its 8 sums per column are added in order through shared memory.
template <typename T, bool RMS, int VL>
__global__ void __launch_bounds__(kColX *kColY)
norm_cols_kernel(const void *__restrict__ x, const void *__restrict__ dy, const float *__restrict__ mean,
                 const float *__restrict__ invstd, float *__restrict__ partial, int64_t rows, int64_t C,
                 int64_t per_slab, unsigned int col_blocks)
{
    using It = Item<T, VL>;
    __shared__ float red[kColY][kColX * VL * 2 + 1];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int items = (int)(C / VL);
    const unsigned int slab = blockIdx.x / col_blocks, col = blockIdx.x % col_blocks;
    const int64_t item = (int64_t)col * kColX + tx;
    const int64_t r0 = (int64_t)slab * per_slab, r1 = r0 + per_slab < rows ? r0 + per_slab : rows;
    float sg[VL] = {}, sb[VL] = {};
    pdl_wait();
    if (item < items) {
        for (int64_t r = r0 + ty; r < r1; r += kColY) {
            const float m = RMS ? 0.f : mean[r], is = invstd[r];
            float f[VL], d[VL];
            It::unpack(It::load(x, r * items + item), f);
            It::unpack(It::load(dy, r * items + item), d);
#pragma unroll
            for (int e = 0; e < VL; ++e) {
                sg[e] = fmaf(d[e], (f[e] - m) * is, sg[e]);
                sb[e] += d[e];
            }
        }
    }
    pdl_trigger();
#pragma unroll
    for (int e = 0; e < VL; ++e) {
        red[ty][tx * VL + e] = sg[e];
        red[ty][kColX * VL + tx * VL + e] = sb[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kColX * VL; i += kColX * kColY) {
        const int half = i / (kColX * VL);
        const int64_t c = (int64_t)col * kColX * VL + i % (kColX * VL);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kColY; ++k) s += red[k][i];
        if (c < C) partial[((int64_t)slab * 2 + half) * C + c] = s;
    }
}

// dgamma[c], dbeta[c]: the slabs' sums in order, in fp64.  16 rows of threads
// to 32 columns, eight loads in flight each.
constexpr int kFinY = 16;
template <typename TP>
__global__ void __launch_bounds__(kColX *kFinY)
norm_finish_kernel(const float *__restrict__ partial, void *__restrict__ dgamma, void *__restrict__ dbeta, int64_t C,
                   int64_t slabs)
{
    __shared__ double red[kFinY][kColX];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * kColX + tx;   // over 2 C: dgamma, then dbeta
    const bool beta = i >= C;
    void *out = beta ? dbeta : dgamma;
    const bool live = i < 2 * C && out;
    pdl_wait();
    double s = 0.0;
    if (live) {
        const float *p = partial + i;
        int64_t k = ty;
        for (; k + 7 * kFinY < slabs; k += 8 * kFinY) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = p[(k + u * kFinY) * 2 * C];
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
        for (; k < slabs; k += kFinY) s += p[k * 2 * C];
    }
    red[ty][tx] = s;
    __syncthreads();
    pdl_trigger();
    if (ty == 0 && live) {
#pragma unroll
        for (int k = 1; k < kFinY; ++k) s += red[k][tx];
        Store<TP>::store1(out, beta ? i - C : i, (float)s);
    }
}

// The backward's ring: R rows of a thread between two barriers (32 elements,
// 16 in fp32: a barrier, its waits and the shuffles of a row sum cost as much
// as the arithmetic of 8), in stages of R S rows.
template <typename T, int VL, int NV>
struct BwdRing {
    static constexpr int kElems = 64 / Store<T>::kBytes;           // of a thread, per stage and tensor
    static constexpr int R = VL * NV >= kElems ? 1 : kElems / (VL * NV) < 4 ? kElems / (VL * NV) : 4;
    static constexpr bool kKeep = VL * NV <= 8;                    // gamma in registers
    static constexpr uint32_t bytes = (uint32_t)kRingThreads * R * NV * VL * Store<T>::kBytes + 32;   // of one tensor
    static constexpr int kFit = (int)((208u << 10) / (2 * bytes));
    static constexpr int stages = kFit < 6 ? kFit : 6;
    static constexpr size_t smem = (size_t)stages * 2 * bytes;
    static_assert(stages >= 3, "a stage in use, one just left and one on its way");
};

// dx and the column sums of one slab of rows in one pass over x and dy: the
// rows' sums, then the results, the elements read twice from the stage.
template <typename T, typename TP, bool RMS, int VL, int NV>
__global__ void __launch_bounds__(kRingThreads, 1)
norm_bwd_ring_kernel(const void *x, const void *dy, const void *__restrict__ gamma, const float *__restrict__ mean_in,
                     const float *__restrict__ invstd_in, void *dx, float *__restrict__ partial, int64_t rows,
                     int64_t C, int G, int S, int64_t per_slab)
{
    using F = BwdRing<T, VL, NV>;
    using V = RingView<T, VL>;
    constexpr int kRing = F::stages, eb = Store<T>::kBytes, R = F::R, N = RMS ? R : 2 * R;
    constexpr uint32_t kBytes = F::bytes;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kRing];
    __shared__ float red[2][N][16];
    const int tid = threadIdx.x, slot = tid / G, g = tid - slot * G, w0 = slot * (G >> 5);
    const int items = (int)(C / VL), SR = S * R;
    const int64_t r0 = (int64_t)blockIdx.x * per_slab, r1 = r0 + per_slab < rows ? r0 + per_slab : rows;
    const int steps = r1 > r0 ? (int)((r1 - r0 + SR - 1) / SR) : 0;
    const float rc = 1.f / (float)C;
    if (tid == 0) {
        for (int s = 0; s < kRing; ++s) mbar_init(smem_addr(full + s), 1);
        mbar_init_fence();
    }
    __syncthreads();
    pdl_wait();
    auto fill = [&](int s, int st) {
        const int64_t a = r0 + (int64_t)s * SR, b = a + SR < r1 ? a + SR : r1;
        const uint32_t bar = smem_addr(full + st), n = V::bytes(a * C, b * C, rows * C);
        unsigned char *dst = ring + st * 2 * kBytes;
        mbar_arrive_expect_tx(bar, 2 * n);
        V::copy(dst, x, a * C, b * C, n, bar);
        V::copy(dst + kBytes, dy, a * C, b * C, n, bar);
    };
    if (tid == 0)
        for (int s = 0; s < kRing && s < steps; ++s) fill(s, s);
    if constexpr (VL == 1) __syncthreads();

    float wk[F::kKeep ? NV : 1][VL], ag[NV][VL], ab[NV][VL];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < VL; ++e) ag[j][e] = ab[j][e] = 0.f;
        if constexpr (F::kKeep)
            if (g + j * G < items) load_params<TP, VL>(gamma, g + j * G, 1.f, wk[j]);
    }
    auto weigh = [&](int j, const float (&d)[VL], float (&p)[VL]) {   // p = d gamma
        if constexpr (F::kKeep) {
            v_mul(d, wk[j], p);
        } else {
            float w[VL];
            load_params<TP, VL>(gamma, g + j * G, 1.f, w);
            v_mul(d, w, p);
        }
    };
    V view(r0, C, SR, slot, g);
    const int row_hop = (int)(S * C);              // elements between a thread's rows of one stage
    const int64_t at0 = ((r0 + slot) * C + g * VL) * eb, hop = (int64_t)SR * C * eb, rh = (int64_t)row_hop * eb;
    unsigned char *op = static_cast<unsigned char *>(dx) + at0;
    float mean_n[R], is_n[R];                      // statistics of the next stage's rows
    const float *mp = RMS ? nullptr : mean_in + r0, *ip = invstd_in + r0;
    const int count = (int)(r1 - r0);              // rows of the slab (below 0 past the end); at: this thread's next
    int at = slot;
    auto stats = [&] {
#pragma unroll
        for (int r = 0; r < R; ++r, at += S) {
            mean_n[r] = RMS || at >= count ? 0.f : mp[at];
            is_n[r] = at >= count ? 0.f : ip[at];
        }
    };
    stats();
    int left = slot < count ? (count - slot + S - 1) / S : 0;   // rows of this slot still to come
    int st = 0;
    uint32_t turn = 0;
    for (int s = 0; s < steps; ++s, op += hop) {
        float mean[R], is[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = mean_n[r];
            is[r] = is_n[r];
        }
        if (!mbar_wait(smem_addr(full) + 8 * st, turn)) atomicExch(&g_norm_error, 1u);
        stats();
        const unsigned char *sx = ring + st * 2 * kBytes, *sd = sx + kBytes;
        const int live = left < R ? left : R;      // this slot's rows in the stage
        left = left < R ? 0 : left - R;
        float v[N];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float t1[2] = {0.f, 0.f}, t2[2] = {0.f, 0.f};
            if (r < live) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (g + j * G < items) {
                        float h[VL], d[VL], p[VL];
                        view.load(sx, j * G, r * row_hop, h);
                        view.load(sd, j * G, r * row_hop, d);
                        if (!RMS) v_shift(h, mean[r]);
                        weigh(j, d, p);
                        if (!RMS) v_sum(p, t1);
                        v_dot(p, h, t2);
                    }
            }
            v[r] = (t2[0] + t2[1]) * is[r];
            if constexpr (!RMS) v[R + r] = t1[0] + t1[1];
        }
        reduce_rows<N>(v, G, w0, &red[s & 1]);
        // every thread has left the stage before this one
        const int prev = st == 0 ? kRing - 1 : st - 1;
        if (tid == 0 && s > 0 && s - 1 + kRing < steps) fill(s - 1 + kRing, prev);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= live) break;
            const float c1 = RMS ? 0.f : -is[r] * (v[N - R + r] * rc), c2 = -is[r] * (v[r] * rc);
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (g + j * G < items) {
                    float h[VL], d[VL], p[VL];
                    view.load(sx, j * G, r * row_hop, h);
                    view.load(sd, j * G, r * row_hop, d);
                    v_center(h, mean[r], is[r]);
                    v_fma(d, h, ag[j]);
                    v_add(d, ab[j]);
                    weigh(j, d, p);
                    v_dx(p, h, is[r], c2, c1);
                    Item<T, VL>::store(op + r * rh, j * G, p);
                }
        }
        if (++st == kRing) {
            st = 0;
            turn ^= 1;
        }
        view.next();
    }
    pdl_trigger();
    if (!partial) return;
    // the S slots' sums of each column, in order
    float *col = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float *out = partial + ((int64_t)blockIdx.x * 2 + half) * C;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (g + j * G < items)
#pragma unroll
                for (int e = 0; e < VL; ++e) {
                    const int c = (g + j * G) * VL + e;
                    const float v = half ? ab[j][e] : ag[j][e];
                    if (S > 1)
                        col[slot * (int)C + c] = v;
                    else
                        out[c] = v;
                }
        if (S == 1) continue;
        __syncthreads();
        for (int c = tid; c < (int)C; c += blockDim.x) {
            float t = 0.f;
            for (int k = 0; k < S; ++k) t += col[k * (int)C + c];
            out[c] = t;
        }
    }
}

// dx of one row per group of threads.  dx may be x or dy itself: every
// element is read before it is written, by the thread that writes it.
template <typename T, typename TP, bool RMS, int VL, int NV>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_dx_kernel(const void *x, const void *dy, const void *__restrict__ gamma, const float *__restrict__ mean_in,
               const float *__restrict__ invstd_in, void *dx, int64_t rows, int64_t C, int lg)
{
    using It = Item<T, VL>;
    __shared__ float red[32];
    const int g = threadIdx.x & ((1 << lg) - 1), G = 1 << lg;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> lg) + (threadIdx.x >> lg);
    const bool live = row < rows;
    const int items = (int)(C / VL);
    const int64_t base = row * items;
    const float rc = 1.f / (float)C;
    pdl_wait();
    typename It::Raw rx[NV], rd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) {
            rx[j] = It::load_rw(x, base + g + j * G);
            rd[j] = It::load_rw(dy, base + g + j * G);
        }
    const float mean = RMS || !live ? 0.f : mean_in[row], is = live ? invstd_in[row] : 0.f;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) {
            float f[VL], d[VL], w[VL];
            It::unpack(rx[j], f);
            It::unpack(rd[j], d);
            load_params<TP, VL>(gamma, g + j * G, 1.f, w);
#pragma unroll
            for (int e = 0; e < VL; ++e) {
                d[e] *= w[e];
                f[e] = d[e] * ((f[e] - mean) * is);
            }
            if (!RMS) s1 += tree_sum(d);
            s2 += tree_sum(f);
        }
    const float m1 = RMS ? 0.f : group_sum(s1, lg, red) * rc, m2 = group_sum(s2, lg, red) * rc;
    pdl_trigger();
    if (!live) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (g + j * G < items) {
            float f[VL], d[VL], w[VL];
            It::unpack(rx[j], f);
            It::unpack(rd[j], d);
            load_params<TP, VL>(gamma, g + j * G, 1.f, w);
#pragma unroll
            for (int e = 0; e < VL; ++e) f[e] = is * (fmaf(-((f[e] - mean) * is), m2, d[e] * w[e]) - m1);
            It::store(dx, base + g + j * G, f);
        }
}

template <typename T, typename TP, bool RMS>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_dx_long_kernel(const void *x, const void *dy, const void *__restrict__ gamma, const float *__restrict__ mean_in,
                    const float *__restrict__ invstd_in, void *dx, int64_t rows, int64_t C)
{
    __shared__ double red[32];
    __shared__ float bc[2];
    const int64_t row = blockIdx.x, base = row * C;
    pdl_wait();
    const float mean = RMS ? 0.f : mean_in[row], is = invstd_in[row];
    double s1 = 0.0, s2 = 0.0;
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float w = gamma ? Store<TP>::load1(gamma, i) : 1.f;
        const float a = Store<T>::load1_rw(dy, base + i) * w;
        s1 += a;
        s2 += a * ((Store<T>::load1_rw(x, base + i) - mean) * is);
    }
    s1 = block_sum(s1, red);
    s2 = block_sum(s2, red);
    if (threadIdx.x == 0) {
        bc[0] = RMS ? 0.f : (float)(s1 / (double)C);
        bc[1] = (float)(s2 / (double)C);
    }
    __syncthreads();
    pdl_trigger();
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float w = gamma ? Store<TP>::load1(gamma, i) : 1.f;
        const float xh = (Store<T>::load1_rw(x, base + i) - mean) * is;
        Store<T>::store1(dx, base + i, is * (fmaf(-xh, bc[1], Store<T>::load1_rw(dy, base + i) * w) - bc[0]));
    }
}

// ------------------------------------------------------------ host side

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A row group's shape: 2^lg threads with nv items each; nv = 0 where a row
// does not fit the registers of a block.
struct Group {
    int lg, nv;
};
// The fewest threads that hold a row (a warp sums by shuffles alone and its
// loads are all in flight at once), but no fewer items in flight on the GPU
// than `rows` allows: with few rows a row is spread over more threads.
inline Group pick_group(int64_t items, int64_t rows, int nv_max)
{
    int nv_want = nv_max;
    while (nv_want > 1 && rows * ((items + nv_want - 1) / nv_want) < (int64_t)kB200Sms * 1024) nv_want >>= 1;
    int lg = 5;
    while (lg < 10 && ((int64_t)nv_want << lg) < items) ++lg;
    int nv = 1;
    while (((int64_t)nv << lg) < items) nv <<= 1;
    return Group{lg, nv <= nv_max ? nv : 0};
}

// A ring kernel's geometry: `want` items per thread where `most_threads` hold
// the row so, more (up to `most`) where they do not; false where no number
// does.
inline bool ring_geo(int64_t items, int want, int most, int most_threads, RingGeo *r)
{
    int nv = 1;
    while (nv < want && nv < items) nv <<= 1;
    while (nv <= most && (items + nv - 1) / nv > most_threads) nv <<= 1;
    if (nv > most) return false;
    const int need = (int)((items + nv - 1) / nv);
    int G = 1;
    while (G < 32 && G < need) G <<= 1;
    if (need > 32) G = (need + 31) / 32 * 32;
    *r = RingGeo{G, most_threads / G, nv};
    return true;
}

template <typename F>
cudaError_t by_nv(int nv, F f)
{
    switch (nv) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    }
    return cudaErrorInvalidValue;
}

template <typename T, typename TP, bool RMS, int VL, int NV>
cudaError_t fwd_ring_nv(const NormLaunch &a, const RingGeo &r)
{
    using F = FwdRing<T, VL, NV>;
    auto kernel = norm_fwd_ring_kernel<T, TP, RMS, VL, NV>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F::smem);
    if (e != cudaSuccess) return e;
    int64_t blocks = (a.rows + r.S - 1) / r.S;
    if (blocks > F::kBlocks * sm_count()) blocks = F::kBlocks * sm_count();
    const int64_t per = (a.rows + blocks - 1) / blocks;
    return launch_pdl(kernel, dim3((unsigned)((a.rows + per - 1) / per)), dim3(r.G * r.S), F::smem, a.stream, a.x,
                      a.gamma, a.beta, a.eps, a.out, a.mean, a.invstd, a.rows, a.C, r.G, r.S, per);
}

// 16 elements of a row per thread, up to 64 (16 one by one) for rows of more
// than 256 threads' worth.  Few rows take the kernel above it: nothing to
// stream, and a row spread over more threads answers sooner.
template <typename T, typename TP, bool RMS, int VL>
bool fwd_ring(const NormLaunch &a, cudaError_t *e)
{
    constexpr int kWant = 16 / VL, kMost = VL == 1 ? 16 : 64 / VL;
    RingGeo r;
    if (a.rows * a.C * Store<T>::kBytes < kRingBytes || !aligned16(a.x) || !ring_geo(a.C / VL, kWant, kMost, kFwdThreads, &r))
        return false;
    *e = by_nv(r.nv, [&](auto n) -> cudaError_t {
        constexpr int NV = decltype(n)::value;
        if constexpr (NV > kMost)
            return cudaErrorInvalidValue;
        else
            return fwd_ring_nv<T, TP, RMS, VL, NV>(a, r);
    });
    return true;
}

// The warp-to-a-row forward: rows of 33 to 512 vectors (below, lanes idle or
// shuffles outweigh the row), and enough of them to give every warp some.
template <typename T, typename TP, bool RMS>
bool fwd_warp(const NormLaunch &a, cudaError_t *e)
{
    const int64_t items = a.C / Store<T>::V, grid = 2 * sm_count();
    if (items <= 32 || items > 512 || a.rows < 2 * kB200Sms * (kWarpThreads / 32)) return false;
    constexpr int kParam = Store<T>::V * Store<TP>::kBytes * 2 < 16 ? 16 : Store<T>::V * Store<TP>::kBytes * 2;
    int nv = 2;
    while (nv * 32 < items) nv <<= 1;
    *e = by_nv(nv, [&](auto n) -> cudaError_t {    // 2 to 16; 512 vectors' parameters are 32 KB
        constexpr int NV = decltype(n)::value;
        if constexpr (NV == 1)
            return cudaErrorInvalidValue;
        else
            return launch_pdl(norm_fwd_warp_kernel<T, TP, RMS, NV>, dim3((unsigned)grid), dim3(kWarpThreads),
                              (size_t)items * kParam, a.stream, a.x, a.gamma, a.beta, a.eps, a.out, a.mean, a.invstd,
                              a.rows, a.C);
    });
    return true;
}

template <typename T, typename TP, bool RMS, int VL>
cudaError_t fwd_vl(const NormLaunch &a)
{
    cudaError_t re;
    if constexpr (VL > 1)
        if (fwd_warp<T, TP, RMS>(a, &re)) return re;
    if (fwd_ring<T, TP, RMS, VL>(a, &re)) return re;
    // 16 vectors a thread in blocks of 256, 8 in blocks of 1024 (64 registers each)
    Group g = pick_group(a.C / VL, a.rows, 16);
    if (VL > 1 && g.nv > 8 && (1 << g.lg) > kNormThreads) g = pick_group(a.C / VL, a.rows, 8);
    if (g.nv == 0)
        return launch_pdl(norm_fwd_long_kernel<T, TP, RMS>, dim3((unsigned)a.rows), dim3(kNormMaxThreads), 0, a.stream,
                          a.x, a.gamma, a.beta, a.eps, a.out, a.mean, a.invstd, a.rows, a.C);
    const int threads = (1 << g.lg) > kNormThreads ? (1 << g.lg) : kNormThreads;
    const int64_t per = threads >> g.lg;
    // Vectors: 2 to 8 a thread are asked for by tensors that the kernels above
    // take, unless the row fills 1024 threads; 16 by bf16 rows of 2049 to 4096
    // vectors in blocks of 256 alone (fp32 rows as long are the ring's).
    constexpr bool kVec = VL > 1;
    return by_nv(g.nv, [&](auto nv) -> cudaError_t {
        constexpr int NV = decltype(nv)::value;
        constexpr bool kWide = !kVec || NV <= 8, kNarrow = !kVec || NV == 1 || (NV == 16 && VL == 8);
        auto launch = [&](auto kernel) {
            return launch_pdl(kernel, dim3((unsigned)((a.rows + per - 1) / per)), dim3(threads), 0, a.stream, a.x,
                              a.gamma, a.beta, a.eps, a.out, a.mean, a.invstd, a.rows, a.C, g.lg);
        };
        if constexpr (kWide)
            if (threads > kNormThreads) return launch(norm_fwd_kernel<T, TP, RMS, VL, NV, kNormMaxThreads>);
        if constexpr (kNarrow)
            if (threads == kNormThreads) return launch(norm_fwd_kernel<T, TP, RMS, VL, NV, kNormThreads>);
        return cudaErrorInvalidValue;
    });
}

template <typename T, typename TP, bool RMS, int VL, int NV>
cudaError_t bwd_ring_nv(const NormLaunch &a, const RingGeo &r)
{
    using F = BwdRing<T, VL, NV>;
    auto kernel = norm_bwd_ring_kernel<T, TP, RMS, VL, NV>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F::smem);
    if (e != cudaSuccess) return e;
    const bool sums = a.dgamma || a.dbeta;
    const int64_t slabs = norm_slabs(a.rows, r.S * F::R), per = (a.rows + slabs - 1) / slabs;
    e = launch_pdl(kernel, dim3((unsigned)slabs), dim3(r.G * r.S), F::smem, a.stream, a.x, a.dy, a.gamma,
                   a.mean_in, a.invstd_in, a.out, static_cast<float *>(sums ? a.workspace : nullptr), a.rows, a.C, r.G,
                   r.S, per);
    if (e != cudaSuccess || !sums) return e;
    return launch_pdl(norm_finish_kernel<TP>, dim3((unsigned)((2 * a.C + kColX - 1) / kColX)), dim3(kColX * kFinY), 0,
                      a.stream, static_cast<const float *>(a.workspace), a.dgamma, a.dbeta, a.C, slabs);
}

// 8 elements of a row per thread, up to 32 (16 one by one) for rows of more
// than 512 threads' worth.
template <typename T, typename TP, bool RMS, int VL>
bool bwd_ring(const NormLaunch &a, cudaError_t *e)
{
    constexpr int kWant = 8 / VL, kMost = (VL == 1 ? 16 : Store<T>::kBytes == 2 ? 32 : 16) / VL;
    RingGeo r;
    if (!aligned16(a.x) || !aligned16(a.dy) || !ring_geo(a.C / VL, kWant, kMost, kRingThreads, &r)) return false;
    *e = by_nv(r.nv, [&](auto n) -> cudaError_t {
        constexpr int NV = decltype(n)::value;
        if constexpr (NV > kMost)
            return cudaErrorInvalidValue;
        else
            return bwd_ring_nv<T, TP, RMS, VL, NV>(a, r);
    });
    return true;
}

template <typename T, typename TP, bool RMS, int VL>
cudaError_t bwd_vl(const NormLaunch &a)
{
    // items per thread of two tensors, in 64 registers; vectors: rows that the
    // ring does not hold give each of 1024 threads three or four
    constexpr int kMost = VL == 1 ? 16 : 4, kLeast = VL == 1 ? 1 : 4;
    cudaError_t fe;
    if (bwd_ring<T, TP, RMS, VL>(a, &fe)) return fe;
    if (a.dgamma || a.dbeta) {
        float *partial = static_cast<float *>(a.workspace);
        const int64_t slabs = norm_slabs(a.rows, kColY), per = (a.rows + slabs - 1) / slabs;
        const int64_t cb = (a.C + kColX * VL - 1) / (kColX * VL);
        cudaError_t e = launch_pdl(norm_cols_kernel<T, RMS, VL>, dim3((unsigned)(cb * slabs)),
                                   dim3(kColX * kColY), 0, a.stream, a.x, a.dy, a.mean_in, a.invstd_in, partial,
                                   a.rows, a.C, per, (unsigned)cb);
        if (e != cudaSuccess) return e;
        e = launch_pdl(norm_finish_kernel<TP>, dim3((unsigned)((2 * a.C + kColX - 1) / kColX)), dim3(kColX * kFinY), 0,
                       a.stream, partial, a.dgamma, a.dbeta, a.C, slabs);
        if (e != cudaSuccess) return e;
    }
    const Group g = pick_group(a.C / VL, a.rows, kMost);
    if (g.nv == 0)
        return launch_pdl(norm_dx_long_kernel<T, TP, RMS>, dim3((unsigned)a.rows), dim3(kNormMaxThreads), 0, a.stream,
                          a.x, a.dy, a.gamma, a.mean_in, a.invstd_in, a.out, a.rows, a.C);
    const int threads = (1 << g.lg) > kNormThreads ? (1 << g.lg) : kNormThreads;
    const int64_t per = threads >> g.lg;
    return by_nv(g.nv, [&](auto nv) -> cudaError_t {
        constexpr int NV = decltype(nv)::value;
        if constexpr (NV < kLeast || NV > kMost)
            return cudaErrorInvalidValue;
        else
            return launch_pdl(norm_dx_kernel<T, TP, RMS, VL, NV>,
                              dim3((unsigned)((a.rows + per - 1) / per)), dim3(threads), 0, a.stream, a.x, a.dy,
                              a.gamma, a.mean_in, a.invstd_in, a.out, a.rows, a.C, g.lg);
    });
}

// Vector items where every row starts on a 16-byte boundary.
template <typename T, typename TP, bool RMS, bool BWD>
cudaError_t by_align(const NormLaunch &a)
{
    constexpr int V = Store<T>::V;
    const bool vec = a.C % V == 0 && aligned16(a.x) && aligned16(a.out) && aligned16(a.gamma) && aligned16(a.beta) &&
                     aligned16(a.dy);
    if constexpr (BWD)
        return vec ? bwd_vl<T, TP, RMS, V>(a) : bwd_vl<T, TP, RMS, 1>(a);
    else
        return vec ? fwd_vl<T, TP, RMS, V>(a) : fwd_vl<T, TP, RMS, 1>(a);
}

template <typename T, typename TP, bool BWD>
cudaError_t by_norm(const NormLaunch &a)
{
    return a.rms ? by_align<T, TP, true, BWD>(a) : by_align<T, TP, false, BWD>(a);
}

template <bool BWD>
cudaError_t by_type(const NormLaunch &a)
{
    if (a.dtype == kBF16) return a.pdtype == kBF16 ? by_norm<Bf16, Bf16, BWD>(a) : by_norm<Bf16, float, BWD>(a);
    return a.pdtype == kBF16 ? by_norm<float, Bf16, BWD>(a) : by_norm<float, float, BWD>(a);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t C)
{
    if (rows <= 0 || C <= 0) return 0;
    return (size_t)norm_slabs(rows, 1) * 2 * (size_t)C * sizeof(float);
}

cudaError_t norm_error_word(int clear, unsigned int *word)
{
    cudaError_t e = cudaMemcpyFromSymbol(word, g_norm_error, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(unsigned int));
    }
    return e;
}

cudaError_t launch_norm_fwd(const NormLaunch &a) { return by_type<false>(a); }
cudaError_t launch_norm_bwd(const NormLaunch &a) { return by_type<true>(a); }

}  // namespace mea
