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
//
// Both are bound by HBM and laid out as the root-mean-square norm's kernels.
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

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// row_reduce of one value: its sum, or its maximum (NaN where there is one).
template <int TPR, int T, bool MAX>
__device__ __forceinline__ float row_reduce1(float a, float *red, int grp) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int sh = W / 2; sh >= 1; sh >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, a, sh);
        a = MAX ? max_nan(a, o) : a + o;
    }
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        if ((threadIdx.x & 31) == 0) red[(threadIdx.x % TPR) >> 5] = a;
        if constexpr (TPR == T) __syncthreads();
        else ptx::named_bar_sync(1 + grp, TPR);
        a = red[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) a = MAX ? max_nan(a, red[w]) : a + red[w];
    }
    return a;
}

template <int DT, int OUT, int TPR, int VPT>
__global__ void __launch_bounds__(norm_threads(TPR)) layernorm_kernel(const LnParams p) {
    constexpr int T = norm_threads(TPR), RPB = T / TPR, NW = TPR > 32 ? TPR / 32 : 1;
    __shared__ float red1[RPB][NW], redm[RPB][NW];
    __shared__ float2 red2[RPB][NW];
    const int grp = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + grp;
    const bool row_ok = row < p.m;
    const int nvec = p.d / 8;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    uint4 xv[VPT], rv[VPT], gv[VPT], bv[VPT];
    const int64_t base = row * p.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        xv[j] = rv[j] = gv[j] = bv[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row_ok && v < nvec) {
            xv[j] = ptx::ld_stream(static_cast<const uint16_t *>(p.x) + base + 8 * v);
            if (p.r != nullptr) rv[j] = ptx::ld_stream(static_cast<const uint16_t *>(p.r) + base + 8 * v);
        }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        if (v < nvec) {
            gv[j] = __ldg(static_cast<const uint4 *>(p.gamma) + v);
            if (p.beta != nullptr) bv[j] = __ldg(static_cast<const uint4 *>(p.beta) + v);
        }
    }
    float s[VPT][8];
    float sum = 0.0f;
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
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += s[j][e];
    }
    const float mu = row_reduce1<TPR, T, false>(sum, red1[grp], grp) * p.inv_d;
    float ss = 0.0f, left = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (j * TPR + t < nvec) {                         // (behind the row's end there is no difference)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[j][e] -= mu;
                ss = fmaf(s[j][e], s[j][e], ss);
                left += s[j][e];
            }
        }
    }
    row_reduce<TPR, T, false>(ss, left, red2[grp], grp);
    left *= p.inv_d;
    const float rho = rsqrtf(fmaxf(fmaf(ss, p.inv_d, -left * left), 0.0f) + p.eps);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float g[8], b[8];
        unpack8<DT>(gv[j], g);
        unpack8<DT>(bv[j], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[j][e] = fmaf((s[j][e] - left) * rho, g[e], b[e]);      // (0 behind the row's end: g and b are)
            if constexpr (OUT != NORM_SAME) top = max_nan(top, fabsf(s[j][e]));
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
        top = row_reduce1<TPR, T, true>(top, redm[grp], grp);
        const bool zero = top <= 1e-35f;
        mul = zero ? 0.0f : C / top;
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
// are held in registers; of longer ones (LONG) the rest is read again, from L2.
template <int DT, int OUT, int TPR, int VPT, bool LONG>
__global__ void __launch_bounds__(norm_threads(TPR)) quant_rows_kernel(const NormParams p) {
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
        float f[8];
        unpack8<DT>(u, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(f[e]));
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) max8(xv[j]);
    if constexpr (LONG)                                   // (one row a block, so the row is there)
        for (int v = VPT * TPR + t; v < nvec; v += TPR) max8(__ldg(reinterpret_cast<const uint4 *>(x + 8 * (int64_t)v)));
    top = row_reduce1<TPR, T, true>(top, red[grp], grp);
    if (!row_ok) return;
    constexpr float C = norm_top_code(OUT);
    const bool zero = top <= 1e-35f;
    const float mul = zero ? 0.0f : C / top;
    if (t == 0) p.scale[row] = zero ? 1.0f : top * (1.0f / C);
    uint8_t *y = static_cast<uint8_t *>(p.y) + row * p.d;
    auto put8 = [&](int v, const uint4 &u) {
        float f[8];
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
// columns, so it has two vectors of a row where that kernel has four, and holds a and s - mu in registers through the two
// reductions; with four vectors (rows beyond 8192) they are taken from the ring again.
constexpr int ln_ring(bool cluster) { return cluster ? 4 : 2; }
constexpr int ln_ring_bytes(int threads, int vpt, bool cluster) { return ln_ring(cluster) * 3 * threads * vpt * 16; }

template <int DT, int TPR, int VPT, bool CLUSTER = false>
__global__ void __launch_bounds__(CLUSTER ? NORM_CLUSTER_T : norm_bwd_threads(TPR, VPT), 1)
    layernorm_bwd_kernel(const LnBwdParams p) {
    constexpr int T = CLUSTER ? NORM_CLUSTER_T : norm_bwd_threads(TPR, VPT), RPB = T / TPR, RING = ln_ring(CLUSTER);
    constexpr int ARRAY = T * VPT;                    // vectors of one array in a stage of the ring
    constexpr int NW = TPR > 32 ? TPR / 32 : 1;
    extern __shared__ uint4 ring[];                   // [RING][dy, s, ds][vector][thread]
    __shared__ float2 red1[RPB][NW], red2[RPB][NW];     // (either is read before the other's next barrier)
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
    float accg[VPT][8], accb[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * TPR + t;
        gv[j] = v < nvec ? __ldg(static_cast<const uint4 *>(p.gamma) + v) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int e = 0; e < 8; ++e) accg[j][e] = accb[j][e] = 0.0f;
    }
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
        float a[HOLD ? VPT : 1][8], c[HOLD ? VPT : 1][8];
        // a and s of vector j
        auto load = [&](int j, float (&av)[8], float (&sv)[8]) {
            float g[8];
            unpack8<DT>(cur[j * T], av);
            unpack8<DT>(cur[ARRAY + j * T], sv);
            unpack8<DT>(gv[j], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) av[e] *= g[e];
        };
        float mu = 0.0f, ma = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (row_ok && j * TPR + t < nvec) {
                float av[8], sv[8];
                load(j, av, sv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mu += sv[e];
                    ma += av[e];
                    if constexpr (HOLD) {
                        a[j][e] = av[e];
                        c[j][e] = sv[e];
                    }
                }
            }
        }
        row_reduce<TPR, T, false>(mu, ma, red1[grp], grp);
        mu *= p.inv_d;
        ma *= p.inv_d;
        float ss = 0.0f, as = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (row_ok && j * TPR + t < nvec) {
                float av[8], sv[8];
                if constexpr (!HOLD) load(j, av, sv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = (HOLD ? c[HOLD ? j : 0][e] : sv[e]) - mu;
                    if constexpr (HOLD) c[j][e] = d;
                    ss = fmaf(d, d, ss);
                    as = fmaf(HOLD ? a[HOLD ? j : 0][e] : av[e], d, as);
                }
            }
        }
        row_reduce<TPR, T, false>(ss, as, red2[grp], grp);
        const float rho = rsqrtf(fmaf(ss, p.inv_d, p.eps));
        const float k = rho * (rho * (as * p.inv_d));     // (rho^2 is beyond fp32 beside the smallest eps)
        uint16_t *out = static_cast<uint16_t *>(p.dx) + row * p.d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * TPR + t;
            if (row_ok && v < nvec) {
                float av[8], sv[8], y[8], o[8];
                if constexpr (!HOLD) load(j, av, sv);
                unpack8<DT>(cur[j * T], y);
                unpack8<DT>(skip ? cur[2 * ARRAY + j * T] : make_uint4(0u, 0u, 0u, 0u), o);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = HOLD ? c[HOLD ? j : 0][e] : sv[e] - mu;
                    const float g = HOLD ? a[HOLD ? j : 0][e] : av[e];
                    accb[j][e] += y[e];
                    accg[j][e] = fmaf(y[e] * rho, d, accg[j][e]);
                    o[e] = fmaf(rho, fmaf(-d, k, g - ma), o[e]);
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
                for (int e = 0; e < 8; ++e) {
                    accg[j][e] += __shfl_xor_sync(0xffffffffu, accg[j][e], sh);
                    accb[j][e] += __shfl_xor_sync(0xffffffffu, accb[j][e], sh);
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
                    to[0] = make_float4(accg[j][4 * h], accg[j][4 * h + 1], accg[j][4 * h + 2], accg[j][4 * h + 3]);
                    to[2 * V * G] = make_float4(accb[j][4 * h], accb[j][4 * h + 1], accb[j][4 * h + 2], accb[j][4 * h + 3]);
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
                o[0] = make_float4(accg[j][0], accg[j][1], accg[j][2], accg[j][3]);
                o[1] = make_float4(accg[j][4], accg[j][5], accg[j][6], accg[j][7]);
                o = reinterpret_cast<float4 *>(part + p.d + 8 * v);
                o[0] = make_float4(accb[j][0], accb[j][1], accb[j][2], accb[j][3]);
                o[1] = make_float4(accb[j][4], accb[j][5], accb[j][6], accb[j][7]);
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
