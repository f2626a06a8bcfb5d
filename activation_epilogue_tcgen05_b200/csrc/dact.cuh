// dact.cuh -- backward of the epilogue D = act(z) + R, z = alpha*A.B + bias:
//     dZ = dD * act'(z),    dbias = the sum of dZ over the axis the bias was broadcast along
// (dR is dD itself).  act'(z) comes from the packed sign mask that the forward wrote
// (RELU_AUX), or from z in the 16-bit type:
//     ReLU   z > 0
//     GELU   Phi(z) + z phi(z), Phi and phi the normal distribution and density
//     tanh   1 / cosh(z)^2
// The sums are taken in fp32 on the unrounded dZ, in an order fixed by the shapes.
//
// Bound by HBM (dD and z read once, dZ written once).  A warp covers 256 columns of a row, a
// lane 8 of them (one 16-byte load); a block of 8 warps covers a strip of 256 columns and a
// run of rows, dealt to its warps in turn.  (Warps side by side, 4 KB of a row together, were
// no faster.)  Column sums stay in a lane's registers over the rows; row sums are one butterfly
// a row.  Either way the block writes fp32 partials, one a run of rows or a strip, that a second
// small kernel adds in order, unless the sums end in the block.  Measured (a copy moves 6.55 TB/s):
// 8192 x 14336 bf16 GELU with dbias 114 us, 6.2 TB/s, tanh 113; from the mask 87 us, 5.6 TB/s; dbias alone 38.6 us, 6.1 TB/s.
#pragma once
#include <cstdint>

#include "rmsnorm.cuh"

namespace gemm_epi {

enum : int { DACT_NONE = 0, DACT_RELU = 1, DACT_RELU_MASK = 2, DACT_GELU = 3, DACT_TANH = 4 };

constexpr int DACT_COLS = 256;      // columns of a strip
constexpr int DACT_WARPS = 8;

struct DactParams {
    int64_t m;
    int n;
    int64_t rows;            // rows of a block's run
    const void *dd, *z;
    const uint8_t *aux;      // the mask's bytes
    int64_t aux_pitch;       // bytes a row
    void *dz;
    void *dbias;             // written at once: by dact_rows_kernel (length m), or of a single run (length n)
    float *partial;          // COL: [run][n]; ROW: [strip][m]; or NULL
};

// GELU'(x) = Phi(x) + x phi(x), Phi and phi the normal distribution and density.  With u = |x| and
// phi(u) = e / sqrt(2 pi), e = exp(-u^2 / 2),
//     GELU'(-u) = e w(u),   GELU'(u) = 1 - e w(u),   w(u) = exp(u^2 / 2) (1 - Phi(u)) - u / sqrt(2 pi),
// so that the left side, which falls to 0 as e does, comes from a product and keeps its digits.  (Phi taken as
// 1/2 - (1/2 - tail) loses a tail below 2^-25, and a tail within 1e-7 absolutely, which is enough for the forward,
// is 7 % off at -5.7 and gives 0 from -6.)  The term beside u / sqrt(2 pi) is a polynomial of degree 5 in
// t = 1 / (c u + 2.498) without a constant, fitted by a linear program to its 64-bit values over 0 <= u <= 16: e w is off
// by at most the larger of 1.8e-7 e and 3.6e-5 of itself (7 % of half an f16 step; two degrees more for 1.4e-7 throughout
// left no registers: 8192 x 14336 134 us for 112).  u is cut off at 16, where e is 0 in fp32, so that an infinite x has its
// side's slope.  All but the cut, the signs and the hardware's reciprocal and exponential is done for two elements at once.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f32x2 gelu_slope(float x0, float x1) {
    constexpr float c = 0.84932180028801907f;                                 // sqrt(log2(e) / 2): e = 2^-(c u)^2
    const f32x2 v = mul2(pair(min_nan(fabsf(x0), 16.0f), min_nan(fabsf(x1), 16.0f)), both(c));
    const float2 den = split(add2(v, both(2.498f))), q = split(mul2(v, v));
    const f32x2 t = pair(rcp_approx(den.x), rcp_approx(den.y));
    f32x2 h = fma2(t, both(20.0101986f), both(-24.893486f));
    h = fma2(t, h, both(0.832031548f));
    h = fma2(t, h, both(-2.2361939f));
    h = fma2(t, h, both(-0.653034389f));
    const f32x2 w = fma2(v, both(2.0f * 0.39894228040143268f / c), mul2(t, h));        // -2 w(u)
    const f32x2 left = mul2(pair(ex2_approx(-q.x), ex2_approx(-q.y)), w);
    const f32x2 side = pair(copysignf(0.5f, x0), copysignf(0.5f, x1));
    return fma2(left, side, add2(side, both(0.5f)));
}

// tanh'(x) = 1 / cosh(x)^2 = 4 e / (1 + e)^2, e = exp(-2 |x|): nothing cancels, so the slope of a saturated
// unit keeps its digits (1 - tanh(x)^2 in fp32 has none left beyond |x| = 8).
__device__ __forceinline__ f32x2 tanh_slope(float x0, float x1) {
    const float2 q = split(mul2(pair(fabsf(x0), fabsf(x1)), both(-2.0f * 1.4426950408889634f)));
    const f32x2 e = pair(ex2_approx(q.x), ex2_approx(q.y));
    const float2 den = split(add2(e, both(1.0f)));
    const f32x2 r = pair(rcp_approx(den.x), rcp_approx(den.y));
    return mul2(mul2(e, both(4.0f)), mul2(r, r));
}

// act'(z) of two neighbouring elements.
template <int ACT>
__device__ __forceinline__ f32x2 slope(float z0, float z1) {
    return ACT == DACT_GELU ? gelu_slope(z0, z1) : tanh_slope(z0, z1);
}

// d *= act'(z) for a lane's eight elements (bits: their mask).
template <int ACT>
__device__ __forceinline__ void through_act(float (&d)[8], const float (&z)[8], uint32_t bits) {
    if constexpr (ACT == DACT_RELU_MASK) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = ((bits >> e) & 1u) ? d[e] : 0.0f;
    } else if constexpr (ACT == DACT_RELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = z[e] > 0.0f ? d[e] : 0.0f;
    } else if constexpr (ACT != DACT_NONE) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 f = split(mul2(pair(d[e], d[e + 1]), slope<ACT>(z[e], z[e + 1])));
            d[e] = f.x;
            d[e + 1] = f.y;
        }
    }
}

// With z to read, rows go through a ring of batches in shared memory, each thread copying its own vectors
// (cp.async, as the norm's backward does): the next batch is on its way while the slopes of one are
// worked out (8192 x 14336 GELU 114 us, loaded where it is used 134).  Without z there is little to work
// out, and a batch is loaded into registers by four blocks an SM instead of three (bias alone 38.6 us,
// through a ring 40.6; 1023 x 4104 from the mask 5.4 us against 7.0).
constexpr int DACT_U = 4;                             // rows of a warp in a batch
constexpr bool dact_reads_z(int act) { return act != DACT_NONE && act != DACT_RELU_MASK; }
// Where a slope is computed, two rows of a batch are worked out at a time: with all four interleaved the constants no longer
// fit the 80 registers that three blocks an SM leave (8192 x 14336 GELU 120 us, two at a time 112).
constexpr bool dact_computes(int act) { return act == DACT_GELU || act == DACT_TANH; }
constexpr int DACT_RING = 2;
constexpr int DACT_SMEM = DACT_RING * 2 * DACT_U * 32 * DACT_WARPS * 16;

template <int DT, int ACT, int AXIS>
__global__ void __launch_bounds__(32 * DACT_WARPS, dact_reads_z(ACT) ? 3 : 4) dact_kernel(const DactParams p) {
    constexpr int T = 32 * DACT_WARPS, U = DACT_U;
    constexpr bool Z = dact_reads_z(ACT), SLOPE = dact_computes(ACT);
    extern __shared__ uint4 ring[];                   // Z: [DACT_RING][U][dd, z][T]
    __shared__ float4 sums[AXIS == AXIS_COL ? 64 * DACT_WARPS : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * DACT_COLS + 8 * lane;
    const bool col_ok = col < p.n;                    // n is a multiple of 8
    const int64_t r0 = (int64_t)blockIdx.y * p.rows, r1 = min(p.m, r0 + p.rows);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    auto fetch = [&](int64_t row, int stage) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = row + u * DACT_WARPS;
            if (i < r1 && col_ok) {
                uint4 *dst = ring + (stage * U + u) * 2 * T + threadIdx.x;
                ptx::cp_async_16(dst, static_cast<const uint16_t *>(p.dd) + i * p.n + col);
                ptx::cp_async_16(dst + T, static_cast<const uint16_t *>(p.z) + i * p.n + col);
            }
        }
        ptx::cp_async_commit();                       // (an empty group keeps the count)
    };
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    int64_t row = r0 + warp;
    constexpr int64_t step = U * DACT_WARPS;
    if constexpr (Z) {
#pragma unroll
        for (int i = 0; i < DACT_RING; ++i) fetch(row + i * step, i);
    }
    int stage = 0;
    for (; row < r1; row += step) {
        uint4 dv[U];
        uint32_t bits[U];
        if constexpr (Z) {
            ptx::cp_async_wait<DACT_RING - 1>();
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = row + u * DACT_WARPS;
                dv[u] = make_uint4(0u, 0u, 0u, 0u);
                bits[u] = 0u;
                if (i < r1 && col_ok) {
                    dv[u] = ptx::ld_stream(static_cast<const uint16_t *>(p.dd) + i * p.n + col);
                    if constexpr (ACT == DACT_RELU_MASK) bits[u] = __ldg(p.aux + i * p.aux_pitch + col / 8);
                }
            }
        }
#pragma unroll (SLOPE ? 2 : U)
        for (int u = 0; u < U; ++u) {
            const int64_t i = row + u * DACT_WARPS;
            const bool ok = i < r1 && col_ok;
            const uint4 *src = ring + (stage * U + u) * 2 * T + threadIdx.x;
            float d[8], z[8];
            if constexpr (Z) {
                unpack8<DT>(ok ? src[0] : make_uint4(0u, 0u, 0u, 0u), d);
                unpack8<DT>(ok ? src[T] : make_uint4(0u, 0u, 0u, 0u), z);
            } else {
                unpack8<DT>(dv[u], d);
            }
            through_act<ACT>(d, z, bits[u]);
            if constexpr (ACT != DACT_NONE) {
                if (ok) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dz) + i * p.n + col) = pack8<DT>(d);
            }
            if constexpr (AXIS == AXIS_COL) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 f = split(add2(pair(acc[e], acc[e + 1]), pair(d[e], d[e + 1])));
                    acc[e] = f.x;
                    acc[e + 1] = f.y;
                }
            } else if (p.partial != nullptr) {
                float s = ((d[0] + d[1]) + (d[2] + d[3])) + ((d[4] + d[5]) + (d[6] + d[7]));
#pragma unroll
                for (int sh = 16; sh >= 1; sh >>= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
                if (lane == 0 && i < r1) p.partial[(int64_t)blockIdx.x * p.m + i] = s;
            }
        }
        if constexpr (Z) {
            fetch(row + DACT_RING * step, stage);
            if (++stage == DACT_RING) stage = 0;
        }
    }
    if constexpr (Z) ptx::cp_async_wait<0>();
    if constexpr (AXIS == AXIS_COL) {
        if (p.partial == nullptr && p.dbias == nullptr) return;
        // the warps' sums, in order: [warp][half of a lane's 8][lane]
        sums[(2 * warp) * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        sums[(2 * warp + 1) * 32 + lane] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        __syncthreads();
        if (threadIdx.x < 64 && col_ok) {             // (threads 32 to 63: the second halves)
            float4 a = sums[threadIdx.x];
#pragma unroll
            for (int w = 1; w < DACT_WARPS; ++w) {
                const float4 b = sums[64 * w + threadIdx.x];
                a.x += b.x;
                a.y += b.y;
                a.z += b.z;
                a.w += b.w;
            }
            if (p.dbias != nullptr)                       // one run: this is the whole sum
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.dbias) + col + 4 * warp) =
                    make_uint2(OutT<DT>::pack(a.x, a.y), OutT<DT>::pack(a.z, a.w));
            else
                reinterpret_cast<float4 *>(p.partial + (int64_t)blockIdx.y * p.n + col)[warp] = a;
        }
    }
}

// The bias along the rows: a block takes DACT_U rows whole, its warps side by side on 2048 columns at a
// time, so that a row's sum ends in the block and dbias is written at once: one launch, no scratch, and one
// butterfly a row instead of one every 256 columns (8192 x 14336 ReLU 106 us against 115, 1023 x 4104 from the
// mask 6.7 us a call from Python against 11.0).  The same ring, along the columns.
template <int DT, int ACT>
__global__ void __launch_bounds__(32 * DACT_WARPS, dact_reads_z(ACT) ? 3 : 4) dact_rows_kernel(const DactParams p) {
    constexpr int T = 32 * DACT_WARPS, U = DACT_U, PASS = DACT_WARPS * DACT_COLS;
    constexpr bool Z = dact_reads_z(ACT), SLOPE = dact_computes(ACT);
    extern __shared__ uint4 ring[];                   // Z: [DACT_RING][U][dd, z][T]
    __shared__ float sums[DACT_WARPS][U];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * U;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint16_t *dd = static_cast<const uint16_t *>(p.dd) + r0 * p.n;
    const uint16_t *zz = Z ? static_cast<const uint16_t *>(p.z) + r0 * p.n : nullptr;
    uint16_t *dz = static_cast<uint16_t *>(p.dz) + r0 * p.n;
    const int rows = (int)min((int64_t)U, p.m - r0);
    auto fetch = [&](int64_t col, int stage) {
        if (col < p.n) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < rows) {
                    uint4 *dst = ring + (stage * U + u) * 2 * T + threadIdx.x;
                    ptx::cp_async_16(dst, dd + (int64_t)u * p.n + col);
                    ptx::cp_async_16(dst + T, zz + (int64_t)u * p.n + col);
                }
            }
        }
        ptx::cp_async_commit();
    };
    float acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u] = 0.0f;
    int64_t col = 8 * threadIdx.x;                    // (n may be within a pass of 2^31)
    if constexpr (Z) {
#pragma unroll
        for (int i = 0; i < DACT_RING; ++i) fetch(col + i * PASS, i);
    }
    int stage = 0;
    for (; col < p.n; col += PASS) {
        uint4 dv[U];
        uint32_t bits[U];
        if constexpr (Z) {
            ptx::cp_async_wait<DACT_RING - 1>();
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                dv[u] = make_uint4(0u, 0u, 0u, 0u);
                bits[u] = 0u;
                if (u < rows) {
                    dv[u] = ptx::ld_stream(dd + (int64_t)u * p.n + col);
                    if constexpr (ACT == DACT_RELU_MASK) bits[u] = __ldg(p.aux + (r0 + u) * p.aux_pitch + col / 8);
                }
            }
        }
        // (two rows at a time; their sums go round, so that each is in its place again after the batch)
#pragma unroll (SLOPE ? 1 : U / 2)
        for (int u0 = 0; u0 < U; u0 += 2) {
            float sum[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int u = u0 + k;
                const uint4 *src = ring + (stage * U + u) * 2 * T + threadIdx.x;
                float d[8], z[8];
                if constexpr (Z) {
                    unpack8<DT>(u < rows ? src[0] : make_uint4(0u, 0u, 0u, 0u), d);
                    unpack8<DT>(u < rows ? src[T] : make_uint4(0u, 0u, 0u, 0u), z);
                } else {
                    unpack8<DT>(dv[u], d);
                }
                through_act<ACT>(d, z, bits[u]);
                if constexpr (ACT != DACT_NONE) {
                    if (u < rows) *reinterpret_cast<uint4 *>(dz + (int64_t)u * p.n + col) = pack8<DT>(d);
                }
                sum[k] = acc[k] + (((d[0] + d[1]) + (d[2] + d[3])) + ((d[4] + d[5]) + (d[6] + d[7])));
            }
#pragma unroll
            for (int k = 0; k < U - 2; ++k) acc[k] = acc[k + 2];
            acc[U - 2] = sum[0];
            acc[U - 1] = sum[1];
        }
        if constexpr (Z) {
            fetch(col + DACT_RING * PASS, stage);
            if (++stage == DACT_RING) stage = 0;
        }
    }
    if constexpr (Z) ptx::cp_async_wait<0>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1) acc[u] += __shfl_xor_sync(0xffffffffu, acc[u], sh);
        if (lane == 0) sums[warp][u] = acc[u];
    }
    __syncthreads();
    if (threadIdx.x < rows) {
        float s = sums[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < DACT_WARPS; ++w) s += sums[w][threadIdx.x];
        const uint32_t v = OutT<DT>::pack(s, 0.0f);
        static_cast<uint16_t *>(p.dbias)[r0 + threadIdx.x] = (uint16_t)v;
    }
}

}  // namespace gemm_epi
