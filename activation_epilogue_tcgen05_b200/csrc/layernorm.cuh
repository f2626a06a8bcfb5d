// layernorm.cuh -- layer norm of the rows of a residual stream, with the residual's addition before it and the
// quantisation after it, and its backward pass; and the quantisation of rows alone.
//
// Forward, for each row i of length d (all arithmetic in fp32):
//     s = x + r                          (r optional; s rounded once, to the 16-bit type, when stored)
//     mu = mean_j s_j,  rho = 1 / sqrt(mean_j (s_j - mu)^2 + eps)
//     y_j = (s_j - mu) rho g_j + b_j     (b optional)
// y goes out as the root-mean-square norm's does (rmsnorm.cuh).  A row's maximum is that of y itself: b keeps it
// from coming out of the reduction of the squares, and it is a third reduction.
// The squares are those of the differences, taken from registers once the mean is known: mean s^2 - mu^2 has no digit left where
// the mean is 2^12 times the deviation.  The differences' own sum, which is what rounding left in mu, is taken
// along and put right (the corrected two-pass sum).
//
// Backward, from dY, the stored sum S, the gain g and the gradient dS that reaches s past the norm:
//     u = (s - mu) rho,  a = dy g
//     dx_j = ds_j + rho (a_j - mean a - u_j mean(a u))         (the gradient of x and of r alike)
//     dg_j = sum_i dy_ij u_ij,  db_j = sum_i dy_ij
// mu, rho, mean a and mean(a u) are taken in two reductions of two sums each; no statistic is kept by the forward pass.
// A mean rounded to fp32 can be many deviations of a nearly constant row away.  The sum is not: 2^13 numbers of 11 bits and one
// binade add up exactly in fp32's 24 (a row of more is added up as two), and if a sum is rounded, values that are far apart are
// in it.  So mu is taken as two numbers, the nearest one, which is subtracted, and the rest of the sum over d by an fma, which joins
// mean(a u) and the fma that makes u.  (Putting mu right by the differences' sum, as the forward pass does, is a third sum in
// the second reduction: 8192 x 4096 with the skip gradient 55.5 us, this 50.3, one rounded mu 49.3.)
//
// Both are laid out as the root-mean-square norm's kernels.  With a residual the forward is bound by HBM: 8192 x 4096 bf16 to e4m3 by
// rows 37.8 us, 6.2 TB/s (a copy moves 6.55); 4096 x 8192 to bf16 42.7 us, 6.3 TB/s.  Without one neither HBM nor the
// issue slots are full (8192 x 4096 to int8 25.4 us, 4.0 TB/s, with 63 % of the slots and 34 % of the warps; to bf16 25.6 us, 5.2 TB/s):
// it is the chain of one row a block, load, sum, sum, maximum, store, with no next row on its way.  18 instructions an element with
// a residual to e4m3, 13 without to 16 bits, in pairs (25 and 30 one by one).
#pragma once
#include <cstdint>

#include "rmsnorm.cuh"

namespace gemm_epi {

struct LnParams : NormParams {
    const void *beta;        // may be NULL
};

struct LnBwdParams : NormBwdParams {     // partial: [grid][dgamma, dbeta][d]
    void *dbeta;             // one cluster: dbeta itself, or NULL
};

__device__ __forceinline__ float halves(f32x2 v) {
    const float2 f = split(v);
    return f.x + f.y;
}

// Waits for a row's threads where there are several warps of them.
template <int TPR, int T>
__device__ __forceinline__ void row_sync(int grp) {
    if constexpr (TPR == T) __syncthreads();
    else ptx::named_bar_sync(1 + grp, TPR);
}

// Sum of a over a row's TPR threads, the same bits in each; red: a float for each of its warps.
template <int TPR, int T>
__device__ __forceinline__ float row_sum(float a, float *red, int grp) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int sh = W / 2; sh >= 1; sh >>= 1) a += __shfl_xor_sync(0xffffffffu, a, sh);
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        if ((threadIdx.x & 31) == 0) red[(threadIdx.x % TPR) >> 5] = a;
        row_sync<TPR, T>(grp);
        const f32x2 *r = reinterpret_cast<const f32x2 *>(red);
        f32x2 s = r[0];
#pragma unroll
        for (int w = 1; w < NW / 2; ++w) s = add2(s, r[w]);
        a = halves(s);
    }
    return a;
}

// The same of two values.  The warps of a long row share the work of the first exchange: their lower lanes go on with a, the
// upper ones with b, which halves the shuffles (two sums of 256 threads cost 27 instructions, by two butterflies and a sum over
// the warps for each 44; every thread has but 16 elements to do); red: a pair for each warp.  TWO: a is the sum over the first
// half of the warps and far that over the second.
template <int TPR, int T, bool TWO = false>
__device__ __forceinline__ void row_sum2(float &a, float &b, f32x2 *red, int grp, float *far = nullptr) {
    if constexpr (TPR <= 32) {
#pragma unroll
        for (int sh = TPR / 2; sh >= 1; sh >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, sh);
            b += __shfl_xor_sync(0xffffffffu, b, sh);
        }
    } else {
        constexpr int NW = TPR / 32;
        const bool upper = (threadIdx.x & 16) != 0;
        float v = upper ? b : a;
        v += __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
        for (int sh = 8; sh >= 1; sh >>= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
        if ((threadIdx.x & 15) == 0) reinterpret_cast<float *>(red)[(threadIdx.x % TPR) >> 4] = v;
        row_sync<TPR, T>(grp);
        const ulonglong2 *r = reinterpret_cast<const ulonglong2 *>(red);
        f32x2 s = add2(r[0].x, r[0].y);
#pragma unroll
        for (int w = 1; w < (TWO ? NW / 4 : NW / 2); ++w) s = add2(s, add2(r[w].x, r[w].y));
        const float2 f = split(s);
        a = f.x;
        b = f.y;
        if constexpr (TWO) {
            s = add2(r[NW / 4].x, r[NW / 4].y);
#pragma unroll
            for (int w = NW / 4 + 1; w < NW / 2; ++w) s = add2(s, add2(r[w].x, r[w].y));
            const float2 g = split(s);
            *far = g.x;
            b += g.y;
        }
    }
}

// The largest of a over a row's threads (NaN where there is one); a >= 0.
template <int TPR, int T>
__device__ __forceinline__ float row_max(float a, float *red, int grp) {
    if constexpr (TPR < 32) {
#pragma unroll
        for (int sh = TPR / 2; sh >= 1; sh >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, sh));
    } else {
        // (the bits of numbers from 0 on order as they do, NaN's above them)
        a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
        if constexpr (TPR > 32) {
            constexpr int NW = TPR / 32;
            if ((threadIdx.x & 31) == 0) red[(threadIdx.x % TPR) >> 5] = a;
            row_sync<TPR, T>(grp);
            a = red[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) a = max_nan(a, red[w]);
        }
    }
    return a;
}

// FULL: rows of exactly 8 TPR VPT elements (the powers of two from 128 on), without a question at each vector whether it is there
// and zeros where it is not: 8192 x 4096 bf16 + residual to e4m3 by rows 38.0 us, 39.4 with them.
// Blocks an SM that the forward kernel is compiled for: 24 warps at 80 registers (the same case, not FULL, 39.4 us; left to itself
// the compiler takes as many and orders them worse, 41.8; 28 and 32 warps spilled in every form, 24 spill 16 to 36 bytes a thread in
// the bf16 forms to 8 bits that are not FULL, of 64 to 256 threads a row), and two blocks of the longest rows' 512 threads
// at 64, which take g and b only where they are used (4096 x 14336 bf16 61 us, by one block at a time 85; with residual
// to e4m3 by rows 71 and 102).
constexpr int ln_blocks(int threads) { return threads >= 512 ? 2 : 768 / threads; }
constexpr bool ln_late(int threads) { return threads >= 512; }

template <int DT, int OUT, int TPR, int VPT, bool FULL>
__global__ void __launch_bounds__(norm_threads(TPR), ln_blocks(norm_threads(TPR))) layernorm_kernel(const LnParams p) {
    constexpr int T = norm_threads(TPR), RPB = T / TPR, NW = TPR > 32 ? TPR / 32 : 1;
    __shared__ __align__(16) float red1[RPB][NW], redm[RPB][NW];
    __shared__ __align__(16) f32x2 red2[RPB][NW];
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + grp;
    const bool row_ok = RPB == 1 || row < p.m;
    const int nvec = FULL ? TPR * VPT : p.d / 8;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    uint4 xv[VPT], rv[VPT];
    const int64_t base = row * p.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        if (RPB > 1 || !FULL) xv[j] = rv[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row_ok && v < nvec) {
            xv[j] = ptx::ld_stream(static_cast<const uint16_t *>(p.x) + base + 8 * v);
            if (p.r != nullptr) rv[j] = ptx::ld_stream(static_cast<const uint16_t *>(p.r) + base + 8 * v);
        }
    }
    f32x2 s[VPT][4];
    f32x2 sum = both(0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        unpack8<DT>(xv[j], s[j]);
        if (p.r != nullptr) {
            f32x2 r[4];
            unpack8<DT>(rv[j], r);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = add2(s[j][e], r[e]);
            const int v = j * TPR + t;
            if (p.s != nullptr && row_ok && v < nvec)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.s) + base + 8 * v) = pack8<DT>(s[j]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = add2(sum, s[j][e]);
    }
    const float mu = row_sum<TPR, T>(halves(sum), red1[grp], grp) * p.inv_d;
    // (g and b, the same for every row, are asked for now: they take the registers that x and r had)
    uint4 gv[VPT], bv[VPT];
    auto load_gb = [&](int j) {
        const int v = j * TPR + t;
        if (!FULL) gv[j] = make_uint4(0u, 0u, 0u, 0u);
        if (v < nvec) gv[j] = __ldg(static_cast<const uint4 *>(p.gamma) + v);
        bv[j] = make_uint4(0u, 0u, 0u, 0u);
        if (v < nvec && p.beta != nullptr) bv[j] = __ldg(static_cast<const uint4 *>(p.beta) + v);
    };
    constexpr bool LATE = ln_late(T);
    if constexpr (!LATE) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) load_gb(j);
    }
    f32x2 ss2 = both(0.0f), left2 = both(0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (j * TPR + t < nvec) {                         // (behind the row's end there is no difference)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[j][e] = add2(s[j][e], both(-mu));
                ss2 = fma2(s[j][e], s[j][e], ss2);
                left2 = add2(left2, s[j][e]);
            }
        }
    }
    float ss = halves(ss2), left = halves(left2);
    row_sum2<TPR, T>(ss, left, red2[grp], grp);
    left *= p.inv_d;
    const float rho = rsqrtf(fmaxf(fmaf(ss, p.inv_d, -left * left), 0.0f) + p.eps);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        f32x2 g[4], b[4];
        if constexpr (LATE) load_gb(j);
        unpack8<DT>(gv[j], g);
        unpack8<DT>(bv[j], b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[j][e] = fma2(mul2(add2(s[j][e], both(-left)), both(rho)), g[e], b[e]);     // (0 behind the row's end: g and b are)
            if constexpr (OUT != NORM_SAME) top = max_abs(top, s[j][e]);
        }
    }
    float mul = 1.0f;
    if constexpr (OUT == NORM_E4M3) {
        mul = per_scale(1.0f, p.scale);
        if (p.amax != nullptr) {
            // as the root-mean-square norm's: one word a warp (rows past the last count for nothing), most only read it
            const unsigned int a = __reduce_max_sync(0xffffffffu, row_ok ? __float_as_uint(top) : 0u);
            if ((threadIdx.x & 31) == 0 && a > *reinterpret_cast<volatile unsigned int *>(p.amax)) atomicMax(p.amax, a);
        }
    } else if constexpr (norm_by_rows(OUT)) {
        constexpr float C = norm_top_code(OUT);
        top = row_max<TPR, T>(top, redm[grp], grp);
        const bool zero = top <= 1e-35f;
        mul = zero ? 0.0f : code_factor<OUT>(top);
        if (t == 0 && row_ok) p.scale[row] = zero ? 1.0f : top * (1.0f / C);
    }
    if (!row_ok) return;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        if (v >= nvec) continue;
        if constexpr (OUT == NORM_SAME)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + base + 8 * v) = pack8<DT>(s[j]);
        else
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.y) + base + 8 * v) = codes8<OUT>(s[j], mul);
    }
}

// Rows quantised with one scale each, without a norm: x -> codes and max |x| / 448 (127).  Rows of up to TPR * VPT vectors
// are held in registers; of longer ones (LONG) the rest is read again, from L2.  Three blocks of 512 threads an SM (40 registers, of
// which 24 to 28 bytes are spilled; 8192 x 14336 to int8 58 us, 6.1 TB/s; two 64), two where the rest is read again (2048 x 32768
// 36 us, one 50).
template <int DT, int OUT, int TPR, int VPT, bool LONG>
__global__ void __launch_bounds__(norm_threads(TPR), TPR >= 512 ? (LONG ? 2 : 3) : 1) quant_rows_kernel(const NormParams p) {
    constexpr int T = norm_threads(TPR), RPB = T / TPR, NW = TPR > 32 ? TPR / 32 : 1;
    __shared__ float red[RPB][NW];
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + grp;
    const bool row_ok = row < p.m;
    const int nvec = p.d / 8;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint16_t *x = static_cast<const uint16_t *>(p.x) + row * p.d;
    uint4 xv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        xv[j] = row_ok && v < nvec ? ptx::ld_stream(x + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
    }
    float top = 0.0f;
    auto max8 = [&](const uint4 &u) {
        f32x2 f[4];
        unpack8<DT>(u, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max_abs(top, f[e]);
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) max8(xv[j]);
    if constexpr (LONG)                                   // (one row a block, so the row is there)
        for (int v = VPT * TPR + t; v < nvec; v += TPR) max8(__ldg(reinterpret_cast<const uint4 *>(x + 8 * (int64_t)v)));
    top = row_max<TPR, T>(top, red[grp], grp);
    if (!row_ok) return;
    constexpr float C = norm_top_code(OUT);
    const bool zero = top <= 1e-35f;
    const float mul = zero ? 0.0f : code_factor<OUT>(top);
    if (t == 0) p.scale[row] = zero ? 1.0f : top * (1.0f / C);
    uint8_t *y = static_cast<uint8_t *>(p.y) + row * p.d;
    auto put8 = [&](int v, const uint4 &u) {
        f32x2 f[4];
        unpack8<DT>(u, f);
        *reinterpret_cast<uint2 *>(y + 8 * (int64_t)v) = codes8<OUT>(f, mul);
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (j * TPR + t < nvec) put8(j * TPR + t, xv[j]);
    if constexpr (LONG)
        for (int v = VPT * TPR + t; v < nvec; v += TPR) put8(v, __ldg(reinterpret_cast<const uint4 *>(x + 8 * (int64_t)v)));
}

// Backward: rows dealt and fetched as by rmsnorm_bwd_kernel.  A thread keeps the sums of both gradients of its
// columns, so it has two vectors of a row where that kernel has four, and holds a and s in registers through the two
// reductions; with three or four vectors they are taken from the ring again.  What bounds it is the chain of a row's two
// reductions, with two rows at a time on an SM: 8192 x 4096 with the skip gradient 45.8 us, 5.9 TB/s, and 4.5 for the second launch;
// 4096 x 8192 (one row at a time) 57, 2340 x 14336 64 of 41 at a copy's rate.  (Three or four rows in the ring, 1024 threads of one
// vector, four rows of 128 threads: none faster.)
constexpr int ln_ring(bool cluster) { return cluster ? 4 : 2; }
constexpr int ln_ring_bytes(int threads, int vpt, bool cluster) { return ln_ring(cluster) * 3 * threads * vpt * 16; }

template <int DT, int TPR, int VPT, int T, bool FULL, bool CLUSTER = false>
__global__ void __launch_bounds__(T, 1) layernorm_bwd_kernel(const LnBwdParams p) {
    constexpr int RPB = T / TPR, RING = ln_ring(CLUSTER);
    constexpr int ARRAY = T * VPT;                    // vectors of one array in a stage of the ring
    constexpr int NW = TPR > 32 ? TPR / 32 : 1;
    extern __shared__ uint4 ring[];                   // [RING][dy, s, ds][vector][thread]
    __shared__ __align__(16) f32x2 red1[RPB][NW], red2[RPB][NW];     // (either is read before the other's next barrier)
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR, nvec = FULL ? TPR * VPT : p.d / 8;
    const bool skip = p.ds != nullptr;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    // (zeros behind a row's end and in the place of rows behind the last: they add nothing to a sum)
    auto fetch = [&](int64_t row, int stage) {
        const int64_t base = row * p.d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * TPR + t;
            uint4 *dst = ring + stage * 3 * ARRAY + j * T + threadIdx.x;
            if (row < p.m && v < nvec) {
                ptx::cp_async_16(dst, static_cast<const uint16_t *>(p.dy) + base + 8 * v);
                ptx::cp_async_16(dst + ARRAY, static_cast<const uint16_t *>(p.s) + base + 8 * v);
                if (skip) ptx::cp_async_16(dst + 2 * ARRAY, static_cast<const uint16_t *>(p.ds) + base + 8 * v);
            } else {
                dst[0] = dst[ARRAY] = dst[2 * ARRAY] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        ptx::cp_async_commit();                       // (an empty group keeps the count)
    };
    uint4 gv[VPT];
    f32x2 accg[VPT][4], accb[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        gv[j] = v < nvec ? __ldg(static_cast<const uint4 *>(p.gamma) + v) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e) accg[j][e] = accb[j][e] = both(0.0f);
    }
    // a row's values behind its sum, or behind the sums over either half of its warps
    constexpr bool TWO = 8 * TPR * VPT > 8192;
    int near = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) near += 8 * (TWO ? min(max(nvec - j * TPR, 0), TPR / 2) : 0);
    const float near_d = (float)(TWO ? near : 8 * nvec), far_d = (float)(8 * nvec - near);
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row0 = (int64_t)blockIdx.x * RPB;
#pragma unroll
    for (int i = 0; i < RING; ++i) fetch(row0 + grp + i * step, i);
    int stage = 0;
    // (every group of a block makes the same number of turns: short rows share a warp's shuffles)
    for (; row0 < p.m; row0 += step) {
        const int64_t row = row0 + grp;
        const bool row_ok = row < p.m;
        ptx::cp_async_wait<RING - 1>();
        const uint4 *cur = ring + stage * 3 * ARRAY + threadIdx.x;
        constexpr bool HOLD = VPT <= 2;
        f32x2 a[HOLD ? VPT : 1][4], c[HOLD ? VPT : 1][4];
        // a and s of vector j
        auto load = [&](int j, f32x2(&av)[4], f32x2(&sv)[4]) {
            f32x2 g[4];
            unpack8<DT>(cur[j * T], av);
            unpack8<DT>(cur[ARRAY + j * T], sv);
            unpack8<DT>(gv[j], g);
#pragma unroll
            for (int e = 0; e < 4; ++e) av[e] = mul2(av[e], g[e]);
        };
        f32x2 mu2 = both(0.0f), ma2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            f32x2 av[4], sv[4];
            load(j, av, sv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mu2 = add2(mu2, sv[e]);
                ma2 = add2(ma2, av[e]);
                if constexpr (HOLD) {
                    a[j][e] = av[e];
                    c[j][e] = sv[e];
                }
            }
        }
        float sum = halves(mu2), far = 0.0f, ma = halves(ma2);
        row_sum2<TPR, T, TWO>(sum, ma, red1[grp], grp, &far);
        ma *= p.inv_d;
        const float mu = (sum + far) * p.inv_d;
        const float rest = p.inv_d * (TWO ? fmaf(-mu, near_d, sum) + fmaf(-mu, far_d, far) : fmaf(-mu, near_d, sum));
        f32x2 ss2 = both(0.0f), as2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (j * TPR + t < nvec) {                     // (behind the row's end there is no difference)
                f32x2 av[4], sv[4];
                if constexpr (!HOLD) load(j, av, sv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 d = add2(HOLD ? c[HOLD ? j : 0][e] : sv[e], both(-mu));
                    if constexpr (HOLD) c[j][e] = d;
                    ss2 = fma2(d, d, ss2);
                    as2 = fma2(HOLD ? a[HOLD ? j : 0][e] : av[e], d, as2);
                }
            }
        }
        float ss = halves(ss2), as = halves(as2);
        row_sum2<TPR, T>(ss, as, red2[grp], grp);
        const float rho = rsqrtf(fmaf(ss, p.inv_d, p.eps));
        const float ku = rho * fmaf(as, p.inv_d, -rest * ma), off = -rest * rho;      // mean(a u)
        uint16_t *out = static_cast<uint16_t *>(p.dx) + row * p.d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * TPR + t;
            if (row_ok && v < nvec) {
                f32x2 av[4], sv[4], y[4], o[4];
                if constexpr (!HOLD) load(j, av, sv);
                unpack8<DT>(cur[j * T], y);
                unpack8<DT>(skip ? cur[2 * ARRAY + j * T] : make_uint4(0u, 0u, 0u, 0u), o);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 d = HOLD ? c[HOLD ? j : 0][e] : add2(sv[e], both(-mu));
                    const f32x2 g = HOLD ? a[HOLD ? j : 0][e] : av[e];
                    accb[j][e] = add2(accb[j][e], y[e]);
                    const f32x2 u = fma2(d, both(rho), both(off));
                    accg[j][e] = fma2(y[e], u, accg[j][e]);
                    o[e] = fma2(both(rho), fma2(u, both(-ku), add2(g, both(-ma))), o[e]);
                }
                *reinterpret_cast<uint4 *>(out + 8 * v) = pack8<DT>(o);
            }
        }
        fetch(row + RING * step, stage);
        if (++stage == RING) stage = 0;
    }
    ptx::cp_async_wait<0>();
    if (!CLUSTER && p.partial == nullptr) return;
    // The block's sums: two rows of d floats, dgamma's and dbeta's, in its partial or, in a cluster, in shared memory behind
    // the groups'.
    constexpr int PART = CLUSTER ? RING * 3 * ARRAY / 2 : 0;
    float *part = CLUSTER ? reinterpret_cast<float *>(ring + PART) : p.partial + (int64_t)blockIdx.x * 2 * p.d;
    if constexpr (RPB > 1) {
        // a warp's groups by butterflies, then the block's through the ring, in order:
        // [gradient][group][half of a vector][vector], so that neighbouring threads are on neighbouring words
#pragma unroll
        for (int sh = TPR; sh < 32; sh <<= 1)
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    accg[j][e] = add2(accg[j][e], __shfl_xor_sync(0xffffffffu, accg[j][e], sh));
                    accb[j][e] = add2(accb[j][e], __shfl_xor_sync(0xffffffffu, accb[j][e], sh));
                }
        constexpr int W = TPR < 32 ? 32 : TPR, G = T / W, V = VPT * TPR;
        float4 *sums = reinterpret_cast<float4 *>(ring);
        static_assert(4 * V * G <= (CLUSTER ? PART : RING * 3 * ARRAY), "the ring holds every group's sums");
        __syncthreads();
        if (threadIdx.x % W < TPR) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 *to = sums + (threadIdx.x / W * 2 + h) * V + j * TPR + t;
                    to[0] = quad(accg[j][2 * h], accg[j][2 * h + 1]);
                    to[2 * V * G] = quad(accb[j][2 * h], accb[j][2 * h + 1]);
                }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 4 * nvec; i += T) {
            const int k = i < 2 * nvec ? 0 : 1, q = i - k * 2 * nvec;       // gradient, quad of its row
            const float4 *src = sums + k * 2 * V * G + (q & 1) * V + (q >> 1);
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
        if constexpr (CLUSTER) __syncthreads();       // the rows of sums lie over other threads' vectors
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * TPR + t;
            if (v < nvec) {
                float4 *o = reinterpret_cast<float4 *>(part + 8 * v);
                o[0] = quad(accg[j][0], accg[j][1]);
                o[1] = quad(accg[j][2], accg[j][3]);
                o = reinterpret_cast<float4 *>(part + p.d + 8 * v);
                o[0] = quad(accb[j][0], accb[j][1]);
                o[1] = quad(accb[j][2], accb[j][3]);
            }
        }
    }
    if constexpr (CLUSTER) {
        static_assert(4 * VPT * TPR <= RING * 3 * ARRAY - PART, "the ring holds the rows of sums behind the groups'");
        ptx::cluster_sync();                          // every block's sums are in its shared memory
        const uint32_t mine = ptx::smem_addr(part);
        for (int i = (int)ptx::cluster_ctarank() + NORM_CLUSTER * threadIdx.x; i < 4 * nvec; i += NORM_CLUSTER * T) {
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
            void *to = i < 2 * nvec ? p.dgamma : p.dbeta;
            if (to != nullptr)
                reinterpret_cast<uint2 *>(to)[i < 2 * nvec ? i : i - 2 * nvec] =
                    make_uint2(OutT<DT>::pack(a.x, a.y), OutT<DT>::pack(a.z, a.w));
        }
        ptx::cluster_sync();                          // no block leaves while another reads its sums
    }
}

}  // namespace gemm_epi
