// rmsnorm.cuh -- root-mean-square norm of the rows of a residual stream, with the
// residual's addition before it and, for the FP8 plans that read its output, the
// quantisation after it; and its backward pass.
//
// Forward, for each row i of length d (all arithmetic in fp32):
//     s = x + r                          (r optional; s rounded once, to the 16-bit type, when stored)
//     rho = 1 / sqrt(mean_j s_j^2 + eps)
//     y_j = s_j rho g_j
// y goes out in the 16-bit type, or in e4m3 as y / scale: with a scale the caller gives for the
// whole tensor (max |y| reported), or with one scale a row, max_j |y_j| / 448 (1 for a row of
// zeros); or in 8-bit integers, with one scale a row, max_j |y_j| / 127.  The row maximum needs no second pass:
// max |y| = rho max |s g|, so the sum of squares and the maximum are reduced together, and
// e4m3(y / scale) = e4m3(s g * 448 / max |s g|).
// The norm is taken of the unrounded fp32 sum: the only roundings are the ones of S and Y.
//
// Backward, from dY, the stored sum S, the gain g and the gradient dS that reaches s past the norm:
//     a = dy g,  c = mean_j(a_j s_j),
//     dx_j = ds_j + rho (a_j - s_j rho^2 c)          (the gradient of x and of r alike)
//     dg_j = sum_i dy_ij s_ij rho_i
// rho is taken again from S in the pass that c needs anyway: no statistic is kept by the forward pass.
//
// Both are bound by HBM: a row is read once, held in registers as fp32 (forward) or in a ring in shared
// memory, from where it is read twice (backward), reduced, and written once.  A row is shared by TPR
// threads, each with VPT vectors of 8 elements (16 bytes at a time, neighbouring threads on neighbouring
// vectors): four vectors a thread, so that a thread has many loads in flight and a block enough work;
// one where the backward has few rows, so that a row is done soonest.
// Measured (a copy moves 6.55 TB/s): 8192 x 4096 bf16 with a residual to e4m3 by rows 36.6 us, 6.4 TB/s;
// 16384 x 8192 bf16 to bf16 159 us, 6.75 TB/s; backward with the skip gradient 8192 x 4096 43.9 us, 6.1 TB/s,
// and 4.5 us for dgamma's second launch; 4096 x 14336 f16 70.4 us, 6.7 TB/s, and 5.5 us.
#pragma once
#include <cstdint>

#include "gemm_tc.cuh"

namespace gemm_epi {

enum : int { NORM_SAME = 0, NORM_E4M3 = 1, NORM_E4M3_ROWS = 2, NORM_I8_ROWS = 4 };
constexpr bool norm_by_rows(int out) { return out == NORM_E4M3_ROWS || out == NORM_I8_ROWS; }
// The largest code of an output with one scale a row.
constexpr float norm_top_code(int out) { return out == NORM_I8_ROWS ? 127.0f : 448.0f; }

struct NormParams {
    int64_t m;
    int d;                   // a multiple of 8 (16 for an e4m3 output)
    float eps, inv_d;
    const void *x, *r;       // r may be NULL
    const void *gamma;
    void *s;                 // may be NULL
    void *y;
    float *scale;            // NORM_E4M3: one float, read; NORM_E4M3_ROWS: m floats, written
    unsigned int *amax;      // NORM_E4M3, may be NULL: max |y| as float bits
};

struct NormBwdParams {
    int64_t m;
    int d;
    float eps, inv_d;
    const void *dy, *s, *gamma, *ds;    // ds may be NULL
    void *dx;
    float *partial;          // [grid][d] sums for dgamma, or NULL
    void *dgamma;            // one cluster: dgamma itself, or NULL
};

template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    using O = OutT<DT>;
    return make_uint4(O::pack(f[0], f[1]), O::pack(f[2], f[3]), O::pack(f[4], f[5]), O::pack(f[6], f[7]));
}

// Eight values in pairs, and back to the 16-bit type.
template <int DT>
__device__ __forceinline__ void unpack8(const uint4 &u, f32x2 (&f)[4]) {
    float v[8];
    unpack8<DT>(u, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = pair(v[2 * e], v[2 * e + 1]);
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const f32x2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = split(f[e]);
        w[e] = OutT<DT>::pack(v.x, v.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float4 quad(f32x2 a, f32x2 b) {
    const float2 x = split(a), y = split(b);
    return make_float4(x.x, x.y, y.x, y.y);
}

// The largest of a and the magnitudes of a pair (NaN where there is one).
__device__ __forceinline__ float max_abs(float a, f32x2 v) {
    const float2 f = split(v);
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(f.x), "f"(f.y));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight values times mul as 8-bit codes of the output type.  Integers (|v mul| below 127.5): 1.5 * 2^23 is added, which
// leaves the integer nearest to the product, ties to even, in the sum's low byte; the sum's is the only rounding.
template <int OUT>
__device__ __forceinline__ uint2 codes8(const f32x2 (&v)[4], float mul) {
    const f32x2 m = both(mul);
    if constexpr (OUT == NORM_I8_ROWS) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = split(fma2(v[e], m, both(12582912.0f)));
            w[e] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040);
        }
        return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __nv_cvt_float2_to_fp8x2(split(mul2(v[e], m)), __NV_SATFINITE, __NV_E4M3);
        return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
}
template <int OUT>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float mul) {
    const f32x2 f[4] = {pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])};
    return codes8<OUT>(f, mul);
}

// What the values of a row whose largest magnitude is top are multiplied by.  127 / top is rounded up: half of the largest
// value is a tie between 63 and 64 and has to go to the even 64.  127 is a prime, so there are other ties only where it divides top's
// digits: in bf16 127 / top is a power of two then, and every code of rows quantised alone is that of the exact quotient;
// in f16 (top 3, 5 ... 15 times 127) a tie goes up, to an odd code half of the time.  A y in fp32 within 2^-16 of a tie may go to
// either side of it.
template <int OUT>
__device__ __forceinline__ float code_factor(float top) {
    return OUT == NORM_I8_ROWS ? __fdiv_ru(127.0f, top) : 448.0f / top;
}

// How two parts of `b` below go together: their sum, the larger, the larger or NaN where there is one.
enum : int { REDUCE_SUM = 0, REDUCE_MAX = 1, REDUCE_MAX_NAN = 2 };
template <int OP>
__device__ __forceinline__ float combine(float a, float b) {
    return OP == REDUCE_MAX ? fmaxf(a, b) : OP == REDUCE_MAX_NAN ? max_nan(a, b) : a + b;
}

// Sum of `a` and combination of `b` over the TPR threads of a row, the same
// bits in each of them.  Rows of up to 32 threads use an xor butterfly (every lane of the warp
// takes part, with whatever row it has); longer ones add their warps' results in warp order, and wait
// for their own TPR threads only (barrier 1 + grp) where a block of T threads has several rows.
template <int TPR, int T, int OP>
__device__ __forceinline__ void row_reduce(float &a, float &b, float2 *red, int grp) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int sh = W / 2; sh >= 1; sh >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, sh);
        b = combine<OP>(b, __shfl_xor_sync(0xffffffffu, b, sh));
    }
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        if ((threadIdx.x & 31) == 0) red[(threadIdx.x % TPR) >> 5] = make_float2(a, b);
        if constexpr (TPR == T) __syncthreads();
        else ptx::named_bar_sync(1 + grp, TPR);
        float2 t = red[0];
        a = t.x;
        b = t.y;
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            t = red[w];
            a += t.x;
            b = combine<OP>(b, t.y);
        }
    }
}

// Threads of a block: one row, or as many short ones as make 128 threads.
constexpr int norm_threads(int tpr) { return tpr > 32 ? tpr : 128; }

template <int DT, int OUT, int TPR, int VPT>
__global__ void __launch_bounds__(norm_threads(TPR)) rmsnorm_kernel(const NormParams p) {
    constexpr int RPB = norm_threads(TPR) / TPR;      // rows of a block
    __shared__ float2 red[RPB][TPR > 32 ? TPR / 32 : 1];
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + grp;
    const bool row_ok = row < p.m;
    const int nvec = p.d / 8;
    // launched as a dependent of the kernel before it: nothing in global memory is touched
    // before that one has completed
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    uint4 xv[VPT], rv[VPT], gv[VPT];
    const int64_t base = row * p.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        xv[j] = rv[j] = gv[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row_ok && v < nvec) {
            xv[j] = ptx::ld_stream(static_cast<const uint16_t *>(p.x) + base + 8 * v);
            if (p.r != nullptr) rv[j] = ptx::ld_stream(static_cast<const uint16_t *>(p.r) + base + 8 * v);
        }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        if (v < nvec) gv[j] = __ldg(static_cast<const uint4 *>(p.gamma) + v);
    }
    float s[VPT][8];
    // int8 codes have no NaN, so the row's scale has to show one: the maximum keeps it (e4m3 codes are NaN themselves)
    constexpr int TOP = OUT == NORM_I8_ROWS ? REDUCE_MAX_NAN : REDUCE_MAX;
    float ss = 0.0f, top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        unpack8<DT>(xv[j], s[j]);
        if (p.r != nullptr) {
            float r[8];
            unpack8<DT>(rv[j], r);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[j][e] += r[e];
            const int v = j * TPR + t;
            if (p.s != nullptr && row_ok && v < nvec)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.s) + base + 8 * v) = pack8<DT>(s[j]);
        }
        float g[8];
        unpack8<DT>(gv[j], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fmaf(s[j][e], s[j][e], ss);
            if constexpr (OUT != NORM_SAME) {
                s[j][e] *= g[e];
                top = combine<TOP>(top, fabsf(s[j][e]));
            }
        }
    }
    row_reduce<TPR, norm_threads(TPR), TOP>(ss, top, red[grp], grp);
    const float rho = rsqrtf(fmaf(ss, p.inv_d, p.eps));
    float mul = rho;
    if constexpr (OUT == NORM_E4M3) {
        mul = per_scale(rho, p.scale);
        if (p.amax != nullptr && (TPR <= 32 || t < 32)) {
            // one word a warp (rows past the last hold zeros); most are below the maximum so far and
            // only read it
            const unsigned int a = __reduce_max_sync(0xffffffffu, __float_as_uint(rho * top));
            if ((threadIdx.x & 31) == 0 && a > *reinterpret_cast<volatile unsigned int *>(p.amax)) atomicMax(p.amax, a);
        }
    } else if constexpr (norm_by_rows(OUT)) {
        // 448 / top overflows below 1.4e-36; such a row is one of zeros in 8 bits at any scale in use
        constexpr float C = norm_top_code(OUT);
        const bool zero = OUT == NORM_I8_ROWS ? top <= 1e-35f : !(top > 1e-35f);
        mul = zero ? (OUT == NORM_I8_ROWS ? 0.0f : rho) : code_factor<OUT>(top);
        if (t == 0 && row_ok) p.scale[row] = zero ? 1.0f : rho * top * (1.0f / C);
    }
    if (!row_ok) return;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        if (v >= nvec) continue;
        if constexpr (OUT == NORM_SAME) {
            float g[8];
            unpack8<DT>(gv[j], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[j][e] = s[j][e] * mul * g[e];
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + base + 8 * v) = pack8<DT>(s[j]);
        } else {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + base + 8 * v) = codes8<OUT>(s[j], mul);
        }
    }
}

// Backward.  Rows are dealt to the blocks' groups of TPR threads round-robin; each thread keeps the
// gain's gradient of its columns in registers over its rows, and the block writes one partial row of
// d floats, its groups added in order.  Which rows a partial holds depends on (m, d) alone, so dgamma
// is the same from run to run.
//
// Each thread copies its own vectors of the next rows into a ring of its own in shared memory
// (cp.async, 16 bytes each) while it works on the present one, so that HBM is never waited for by
// all of an SM's threads at once, nothing has to be held in registers across the reduction (the
// second pass reads shared memory again), and no barrier guards the ring: nobody else reads it.
constexpr int NORM_RING = 2;                          // rows of a group in the ring
constexpr int norm_ring_bytes(int threads, int vpt) { return NORM_RING * 3 * threads * vpt * 16; }
// Four vectors a thread: one block of 512 threads an SM, so that there are few partial rows to add up
// (148; with blocks of 128 threads, 592 of them made the second launch 3 us longer at d = 4096).
// One vector a thread (few rows): blocks of one row or 128 threads, again one an SM.
constexpr int norm_bwd_threads(int tpr, int vpt) { return vpt == 1 ? norm_threads(tpr) : 512; }
constexpr int NORM_BWD_BLOCKS = 148;                  // a B200's SMs
// So few rows that one cluster of 8 blocks (512 threads each, one vector a thread) takes them in two turns:
// it adds its blocks' sums through distributed shared memory and writes dgamma itself, in one launch
// and without scratch.  What that saves is the host's and the scratch: a call from Python takes 6.7 us, with
// partial rows and a second launch 9.2 (scratch given; 11.0 with torch's allocator).  On the device, in a
// graph, it is the slower form at most sizes: one turn 4.6 us against 3.9 (8 x 4096), 3.1 and 3.1 (32 x 1024), 2.6 and
// 3.1 (128 x 256); two 5.4 against 4.0 (16 x 4096), 3.8 and 3.1 (64 x 1024), 3.4 and 3.0 (256 x 256, 1024 x 64); four would be
// 6.9 against 4.5 (32 x 4096), 5.1 and 3.6 (128 x 1024).  So two turns are the limit: there the host's saving is still
// above the device's loss.
constexpr int NORM_CLUSTER = 8;
constexpr int NORM_CLUSTER_T = 512;

template <int DT, int TPR, int VPT, bool CLUSTER = false>
__global__ void __launch_bounds__(CLUSTER ? NORM_CLUSTER_T : norm_bwd_threads(TPR, VPT), 1)
    rmsnorm_bwd_kernel(const NormBwdParams p) {
    constexpr int T = CLUSTER ? NORM_CLUSTER_T : norm_bwd_threads(TPR, VPT), RPB = T / TPR;
    constexpr int ARRAY = T * VPT;                    // vectors of one array in a stage of the ring
    extern __shared__ uint4 ring[];                   // [NORM_RING][dy, s, ds][vector][thread]
    __shared__ float2 red[2][RPB][TPR > 32 ? TPR / 32 : 1];
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR, nvec = p.d / 8;
    const bool skip = p.ds != nullptr;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    auto fetch = [&](int64_t row, int stage) {
        if (row < p.m) {
            const int64_t base = row * p.d;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = j * TPR + t;
                if (v < nvec) {
                    uint4 *dst = ring + stage * 3 * ARRAY + j * T + threadIdx.x;
                    ptx::cp_async_16(dst, static_cast<const uint16_t *>(p.dy) + base + 8 * v);
                    ptx::cp_async_16(dst + ARRAY, static_cast<const uint16_t *>(p.s) + base + 8 * v);
                    if (skip) ptx::cp_async_16(dst + 2 * ARRAY, static_cast<const uint16_t *>(p.ds) + base + 8 * v);
                }
            }
        }
        ptx::cp_async_commit();                       // (an empty group keeps the count)
    };
    uint4 gv[VPT];
    float acc[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        gv[j] = v < nvec ? __ldg(static_cast<const uint4 *>(p.gamma) + v) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[j][e] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row0 = (int64_t)blockIdx.x * RPB;
#pragma unroll
    for (int i = 0; i < NORM_RING; ++i) fetch(row0 + grp + i * step, i);
    int stage = 0;
    // (every group of a block makes the same number of turns: short rows share a warp's shuffles)
    for (int buf = 0; row0 < p.m; row0 += step, buf ^= 1) {
        const int64_t row = row0 + grp;
        const bool row_ok = row < p.m;
        ptx::cp_async_wait<NORM_RING - 1>();
        const uint4 *cur = ring + stage * 3 * ARRAY + threadIdx.x;
        float ss = 0.0f, c = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (row_ok && j * TPR + t < nvec) {
                float y[8], s[8], g[8];
                unpack8<DT>(cur[j * T], y);
                unpack8<DT>(cur[ARRAY + j * T], s);
                unpack8<DT>(gv[j], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(s[e], s[e], ss);
                    c = fmaf(y[e] * g[e], s[e], c);
                }
            }
        }
        row_reduce<TPR, T, REDUCE_SUM>(ss, c, red[buf][grp], grp);
        const float rho = rsqrtf(fmaf(ss, p.inv_d, p.eps));
        const float k = rho * (rho * (c * p.inv_d));      // (rho^2 is beyond fp32 beside the smallest eps)
        uint16_t *out = static_cast<uint16_t *>(p.dx) + row * p.d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * TPR + t;
            if (row_ok && v < nvec) {
                float y[8], s[8], g[8], o[8];
                unpack8<DT>(cur[j * T], y);
                unpack8<DT>(cur[ARRAY + j * T], s);
                unpack8<DT>(gv[j], g);
                unpack8<DT>(skip ? cur[2 * ARRAY + j * T] : make_uint4(0u, 0u, 0u, 0u), o);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    acc[j][e] = fmaf(y[e] * rho, s[e], acc[j][e]);
                    o[e] = fmaf(rho, fmaf(-s[e], k, y[e] * g[e]), o[e]);
                }
                *reinterpret_cast<uint4 *>(out + 8 * v) = pack8<DT>(o);
            }
        }
        fetch(row + NORM_RING * step, stage);
        if (++stage == NORM_RING) stage = 0;
    }
    ptx::cp_async_wait<0>();
    if (!CLUSTER && p.partial == nullptr) return;
    // (a cluster's block keeps its row of sums in shared memory, behind the groups')
    constexpr int PART = CLUSTER ? NORM_RING * 3 * ARRAY / 2 : 0;
    float *part = CLUSTER ? reinterpret_cast<float *>(ring + PART) : p.partial + (int64_t)blockIdx.x * p.d;
    if constexpr (RPB > 1) {
        // a warp's groups by butterflies, then the block's through the ring, in order:
        // [group][half of a vector][vector], so that neighbouring threads are on neighbouring words
#pragma unroll
        for (int sh = TPR; sh < 32; sh <<= 1)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[j][e] += __shfl_xor_sync(0xffffffffu, acc[j][e], sh);
        constexpr int W = TPR < 32 ? 32 : TPR, G = T / W, V = VPT * TPR;
        float4 *sums = reinterpret_cast<float4 *>(ring);
        static_assert(2 * V * G <= (CLUSTER ? PART : NORM_RING * 3 * ARRAY), "the ring holds every group's sums");
        __syncthreads();
        if (threadIdx.x % W < TPR) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sums[(threadIdx.x / W * 2 + h) * V + j * TPR + t] =
                        make_float4(acc[j][4 * h], acc[j][4 * h + 1], acc[j][4 * h + 2], acc[j][4 * h + 3]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * nvec; i += T) {
            const float4 *src = sums + (i & 1) * V + (i >> 1);
            float4 a = src[0];
#pragma unroll
            for (int g = 1; g < G; ++g) {
                const float4 b = src[2 * V * g];
                a.x += b.x;
                a.y += b.y;
                a.z += b.z;
                a.w += b.w;
            }
            reinterpret_cast<float4 *>(part)[i] = a;
        }
    } else {
        if constexpr (CLUSTER) __syncthreads();       // the row of sums lies over other threads' vectors
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * TPR + t;
            if (v < nvec) {
                float4 *o = reinterpret_cast<float4 *>(part + 8 * v);
                o[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
                o[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
            }
        }
    }
    if constexpr (CLUSTER) {
        static_assert(2 * VPT * TPR <= NORM_RING * 3 * ARRAY - PART, "the ring holds a row of sums behind the groups'");
        ptx::cluster_sync();                          // every block's sums are in its shared memory
        const uint32_t mine = ptx::smem_addr(part);
        for (int i = (int)ptx::cluster_ctarank() + NORM_CLUSTER * threadIdx.x; i < 2 * nvec; i += NORM_CLUSTER * T) {
            float4 v[NORM_CLUSTER];
#pragma unroll
            for (int b = 0; b < NORM_CLUSTER; ++b) v[b] = ptx::ld_cluster_v4(ptx::mapa(mine + 16u * i, b));
            float4 a = v[0];
#pragma unroll
            for (int b = 1; b < NORM_CLUSTER; ++b) {
                a.x += v[b].x;
                a.y += v[b].y;
                a.z += v[b].z;
                a.w += v[b].w;
            }
            reinterpret_cast<uint2 *>(p.dgamma)[i] = make_uint2(OutT<DT>::pack(a.x, a.y), OutT<DT>::pack(a.z, a.w));
        }
        ptx::cluster_sync();                          // no block leaves while another reads its sums
    }
}

// out[i] = sum_p src[p * len + i] over fp32 partials, len a multiple of 8; from i = cut on (a multiple of 4) the sums go to
// out2[i - cut], and to neither array where its pointer is NULL.  A block takes 32 outputs:
// thread (x, y) adds parts y, y + Y, ... of four neighbouring outputs, ten loads in flight (it is
// latency that counts here: all of a thread's loads should go out at once), then the Y sums are added in
// a fixed tree; the order depends on (parts, len) alone.
template <int DT, int Y>
__global__ void __launch_bounds__(8 * Y) add_parts_kernel(const float *__restrict__ src, int64_t parts, int64_t len,
                                                          void *out, void *out2, int64_t cut) {
    constexpr int U = 10;
    __shared__ float4 red[Y][8];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int64_t i = (int64_t)blockIdx.x * 32 + 4 * x;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < len) {
        const float4 *s4 = reinterpret_cast<const float4 *>(src + i);
        const int64_t pitch = len / 4;
        for (int64_t p0 = y; p0 < parts; p0 += U * Y) {
            float4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = p0 + Y * u < parts ? __ldcg(s4 + (p0 + Y * u) * pitch) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a.x += v[u].x;
                a.y += v[u].y;
                a.z += v[u].z;
                a.w += v[u].w;
            }
        }
    }
    red[y][x] = a;
    __syncthreads();
    // a warp an output quad: Y / 32 of its sums a lane, then a butterfly over the lanes
    const int q = threadIdx.x >> 5, l = threadIdx.x & 31;
    if (q < 8) {
        float4 s = red[l][q];
#pragma unroll
        for (int k = 1; k < Y / 32; ++k) {
            const float4 b = red[l + 32 * k][q];
            s.x += b.x;
            s.y += b.y;
            s.z += b.z;
            s.w += b.w;
        }
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, sh);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, sh);
            s.z += __shfl_xor_sync(0xffffffffu, s.z, sh);
            s.w += __shfl_xor_sync(0xffffffffu, s.w, sh);
        }
        const int64_t o = (int64_t)blockIdx.x * 32 + 4 * q;
        uint16_t *to = o < cut ? static_cast<uint16_t *>(out) : static_cast<uint16_t *>(out2);
        if (l == 0 && o < len && to != nullptr)
            *reinterpret_cast<uint2 *>(to + (o < cut ? o : o - cut)) =
                make_uint2(OutT<DT>::pack(s.x, s.y), OutT<DT>::pack(s.z, s.w));
    }
}

}  // namespace gemm_epi
