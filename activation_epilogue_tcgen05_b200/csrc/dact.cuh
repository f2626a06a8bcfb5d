// dact.cuh -- backward of the epilogue D = act(z) + R, z = alpha*A.B + bias:
//     dZ = dD * act'(z),    dbias = the sum of dZ over the axis the bias was broadcast along
// (dR is dD itself).  act'(z) comes from the packed sign mask that the forward wrote
// (RELU_AUX), or from z in the 16-bit type:
//     ReLU   z > 0
//     GELU   Phi(z) + z phi(z), Phi and phi the normal distribution and density
//     tanh   1 - tanh(z)^2
// The sums are taken in fp32 on the unrounded dZ, in an order fixed by the shapes.
//
// Bound by HBM (dD and z read once, dZ written once).  A warp covers 256 columns of a row, a
// lane 8 of them (one 16-byte load); a block of 8 warps covers a strip of 256 columns and a
// run of rows, dealt to its warps in turn.  Column sums stay in a lane's registers over the
// rows; row sums are one butterfly a row.  Either way the block writes fp32 partials, one a
// strip or a run of rows, that a second small kernel adds in order.
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
    float *partial;          // COL: [run][n]; ROW: [strip][m]; or NULL
};

// GELU's slope takes 27 instructions an element one by one and 14 in pairs, below what HBM allows
// time for.
// GELU'(x) = Phi(x) + x phi(x), with 1 - Phi(|x|) from the same Abramowitz & Stegun 7.1.26 form as
// the forward epilogue's GELU (gelu_erf): one exponential serves both terms.
//     Phi(x) = 1/2 + sign(x) (1/2 - tail),  tail = 1 - Phi(|x|)
__device__ __forceinline__ f32x2 gelu_slope(float x0, float x1) {
    const f32x2 x = pair(x0, x1);
    const float2 den = split(fma2(pair(fabsf(x0), fabsf(x1)), both(0.3275911f * 0.70710678118654752f), both(1.0f)));
    const f32x2 t = pair(rcp_approx(den.x), rcp_approx(den.y));
    f32x2 h = fma2(t, both(0.5307027145f), both(-0.7265760135f));
    h = fma2(t, h, both(0.7107068705f));
    h = fma2(t, h, both(-0.142248368f));
    h = fma2(t, h, both(0.127414796f));
    h = mul2(t, h);
    const f32x2 s = mul2(x, both(0.84932180028801907f));        // (c x)^2 = x^2 / 2 * log2(e)
    const float2 q = split(mul2(s, s));
    const f32x2 e = pair(ex2_approx(-q.x), ex2_approx(-q.y));     // exp(-x^2 / 2)
    const float2 half = split(fma2(mul2(h, both(-1.0f)), e, both(0.5f)));
    const f32x2 phi = pair(copysignf(half.x, x0), copysignf(half.y, x1));
    return add2(fma2(mul2(x, both(0.39894228040143268f)), e, phi), both(0.5f));
}

// act'(z) of two neighbouring elements.
template <int ACT>
__device__ __forceinline__ f32x2 slope(float z0, float z1) {
    if constexpr (ACT == DACT_GELU) {
        return gelu_slope(z0, z1);
    } else {
        const float y0 = tanhf(z0), y1 = tanhf(z1);
        return pair(fmaf(-y0, y0, 1.0f), fmaf(-y1, y1, 1.0f));
    }
}

template <int DT, int ACT, int AXIS>
__global__ void __launch_bounds__(32 * DACT_WARPS, 4) dact_kernel(const DactParams p) {
    __shared__ float sums[DACT_WARPS][DACT_COLS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * DACT_COLS + 8 * lane;
    const bool col_ok = col < p.n;                    // n is a multiple of 8
    const int64_t r0 = (int64_t)blockIdx.y * p.rows, r1 = min(p.m, r0 + p.rows);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    constexpr int U = 4;                              // rows of a warp in flight
    for (int64_t row = r0 + warp; row < r1; row += U * DACT_WARPS) {
        uint4 dv[U], zv[U];
        uint32_t mv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = row + u * DACT_WARPS;
            dv[u] = zv[u] = make_uint4(0u, 0u, 0u, 0u);
            mv[u] = 0u;
            if (i < r1 && col_ok) {
                dv[u] = ptx::ld_stream(static_cast<const uint16_t *>(p.dd) + i * p.n + col);
                if constexpr (ACT == DACT_RELU_MASK) mv[u] = __ldg(p.aux + i * p.aux_pitch + col / 8);
                else if constexpr (ACT != DACT_NONE) zv[u] = ptx::ld_stream(static_cast<const uint16_t *>(p.z) + i * p.n + col);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = row + u * DACT_WARPS;
            float d[8], z[8];
            unpack8<DT>(dv[u], d);
            if constexpr (ACT == DACT_RELU_MASK) {
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = ((mv[u] >> e) & 1u) ? d[e] : 0.0f;
            } else if constexpr (ACT == DACT_RELU) {
                unpack8<DT>(zv[u], z);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = z[e] > 0.0f ? d[e] : 0.0f;
            } else if constexpr (ACT != DACT_NONE) {
                unpack8<DT>(zv[u], z);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 f = split(mul2(pair(d[e], d[e + 1]), slope<ACT>(z[e], z[e + 1])));
                    d[e] = f.x;
                    d[e + 1] = f.y;
                }
            }
            if constexpr (ACT != DACT_NONE) {
                if (i < r1 && col_ok)
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dz) + i * p.n + col) = pack8<DT>(d);
            }
            if constexpr (AXIS == AXIS_COL) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += d[e];
            } else if (p.partial != nullptr) {
                float s = ((d[0] + d[1]) + (d[2] + d[3])) + ((d[4] + d[5]) + (d[6] + d[7]));
#pragma unroll
                for (int sh = 16; sh >= 1; sh >>= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
                if (lane == 0 && i < r1) p.partial[(int64_t)blockIdx.x * p.m + i] = s;
            }
        }
    }
    if constexpr (AXIS == AXIS_COL) {
        if (p.partial == nullptr) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[warp][8 * lane + e] = acc[e];
        __syncthreads();
        const int c = blockIdx.x * DACT_COLS + threadIdx.x;
        float s = sums[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < DACT_WARPS; ++w) s += sums[w][threadIdx.x];
        if (c < p.n) p.partial[(int64_t)blockIdx.y * p.n + c] = s;
    }
}

}  // namespace gemm_epi
