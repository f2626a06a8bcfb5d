// ckpt.cuh -- checkpoints of pre-activations in 8 bits: what the backward pass of an epilogue needs of z, kept in half
// the memory.
//
// 32 neighbouring columns of a row share a power of two (the block format MXINT8 of the OCP Microscaling Formats
// specification: 8-bit integers in units of 2^-6 and one exponent byte, 8 bits and a quarter an element):
//     z ~ q 2^(e - 133),   q = round(z 2^(133 - e)) to nearest, ties to even, in -127 ... 127,
//     e the smallest exponent from 7 on with max |z| <= 127 * 2^(e - 133);
// e = 255 stands for a group with a value that is not finite (or above 127 * 2^121): all of it is restored as NaN.
// With a power of two the products are exact: the codes do not depend on how the quotient is taken, and a code times its step
// is a bf16 number.  The step is between 1/127 and 1/63.5 of the largest magnitude, where bf16's is between 1/256 and 1/128.
//
// save: H = act(z) (the next product's operand, optional), codes and exponents in one pass over z;
// load: z, or act(z), in the 16-bit type again.  Bound by HBM.  A thread takes eight columns, four neighbours a group, so that a
// group's maximum is two shuffles; the groups of all rows are dealt to the threads in one line, so that narrow and
// ragged rows leave few of them idle; U groups a thread, all loads first.
// Measured (a copy moves 6.55 TB/s): 8192 x 14336 bf16 GELU saved in 99 us, 6.0 TB/s (20 instructions an element, three quarters of
// the issue slots), loaded in 52.6, 6.8 TB/s; 32768 x 128 5.2 and 3.2.
#pragma once
#include <cstdint>

#include "rmsnorm.cuh"

namespace gemm_epi {

constexpr int CKPT_GROUP = 32;
constexpr int CKPT_T = 256;
__host__ __device__ constexpr int ckpt_groups(int64_t n) { return (int)((n + CKPT_GROUP - 1) / CKPT_GROUP); }

struct CkptParams {
    int n;
    uint32_t groups;         // of a row
    uint32_t total;          // of all rows
    const void *z;           // save: read
    void *h;                 // save: act(z), or NULL; load: written
    int8_t *codes;
    uint8_t *exps;
};

// The exponent of a group whose largest magnitude has these bits (of a float, without its sign; NaN is above all).  The
// largest code is 127 = 64 * 1.984375, so a mantissa above that takes the next power of two.
__device__ __forceinline__ uint32_t ckpt_exponent(uint32_t top) { return min(max((top + 0x1FFFFu) >> 23, 7u), 255u); }
// 2^(e - 133) and its inverse, e in 7 ... 254 (step: NaN for 255).
__device__ __forceinline__ float ckpt_step(uint32_t e) {
    return e >= 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((max(e, 6u) - 6u) << 23);
}
__device__ __forceinline__ float ckpt_inverse(uint32_t e) { return __uint_as_float((260u - e) << 23); }

// Eight codes -> values.  A byte with its sign flipped, in the low bits of 2^23, is 2^23 + 128 + q.
__device__ __forceinline__ void ckpt_decode8(const uint2 &q, float step, f32x2 (&f)[4]) {
    const f32x2 off = both(-8388736.0f), s = both(step);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t w = (h ? q.y : q.x) ^ 0x80808080u;
        f[2 * h] = pair(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)), __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441)));
        f[2 * h + 1] = pair(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)), __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443)));
        f[2 * h] = mul2(add2(f[2 * h], off), s);
        f[2 * h + 1] = mul2(add2(f[2 * h + 1], off), s);
    }
}

// tanh of two values: (1 - e) / (1 + e), e = exp(-2 |x|), whose numerator is within 2^-23 of it, and x - x^3 / 3 below 1/32,
// where that would show (the next term is x^5 2 / 15 < 2^-22.9 x).
__device__ __forceinline__ f32x2 tanh2(float x0, float x1) {
    const f32x2 x = pair(x0, x1);
    const float2 q = split(mul2(pair(fabsf(x0), fabsf(x1)), both(-2.0f * 1.4426950408889634f)));
    const f32x2 e = pair(ex2_approx(q.x), ex2_approx(q.y));
    const float2 den = split(add2(e, both(1.0f)));
    const float2 big = split(mul2(fma2(e, both(-1.0f), both(1.0f)), pair(rcp_approx(den.x), rcp_approx(den.y))));
    const float2 small = split(fma2(mul2(mul2(x, x), both(-1.0f / 3.0f)), x, x));
    return pair(fabsf(x0) < 0.03125f ? small.x : copysignf(big.x, x0), fabsf(x1) < 0.03125f ? small.y : copysignf(big.y, x1));
}

// act of a thread's eight values.
template <int EPI>
__device__ __forceinline__ void ckpt_act8(f32x2 (&f)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = split(f[e]);
        if constexpr (EPI == EPI_GELU) {
            const float2 y = gelu_erf2(x.x, x.y);
            f[e] = pair(y.x, y.y);
        } else if constexpr (EPI == EPI_TANH) {
            f[e] = tanh2(x.x, x.y);
        } else if constexpr (EPI == EPI_RELU) {
            f[e] = pair(x.x < 0.0f ? 0.0f : x.x, x.y < 0.0f ? 0.0f : x.y);
        }
    }
}

// f16: the kept z of a value near the type's largest number is above it (65536: save's z was rounded up in its step), and so is act
// of it but for tanh's; it is drawn back, in groups whose 127 steps reach that far.  NaN stays NaN.
template <int DT>
__device__ __forceinline__ void ckpt_draw_back8(f32x2 (&f)[4], uint32_t ex) {
    if (DT == DT_F16 && ex >= 143u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x = split(f[e]);
            f[e] = pair(x.x > 65504.0f ? 65504.0f : x.x < -65504.0f ? -65504.0f : x.x,
                        x.y > 65504.0f ? 65504.0f : x.y < -65504.0f ? -65504.0f : x.y);
        }
    }
}

// Where a thread's groups lie: group `id` of all rows, and from it every CKPT_T / 4 further.
struct CkptWalk {
    uint32_t id, row, g, drow, dg;
    __device__ __forceinline__ CkptWalk(const CkptParams &p, int u) {
        id = blockIdx.x * (uint32_t)(CKPT_T / 4 * u) + threadIdx.x / 4;
        row = id / p.groups;
        g = id - row * p.groups;
        drow = (CKPT_T / 4) / p.groups;
        dg = (CKPT_T / 4) - drow * p.groups;
    }
    __device__ __forceinline__ int col() const { return (int)g * CKPT_GROUP + 8 * (threadIdx.x & 3); }
    __device__ __forceinline__ void next(const CkptParams &p) {
        id += CKPT_T / 4;
        row += drow;
        g += dg;
        if (g >= p.groups) {
            g -= p.groups;
            ++row;
        }
    }
};

template <int DT, int EPI, int U>
__global__ void __launch_bounds__(CKPT_T) ckpt_save_kernel(const CkptParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    uint4 zv[U];
    int64_t at[U];                               // the thread's first element; negative: none
    uint32_t id0;
    {
        CkptWalk w(p, U);
        id0 = w.id;
#pragma unroll
        for (int u = 0; u < U; ++u, w.next(p)) {
            at[u] = w.id < p.total && w.col() < p.n ? (int64_t)w.row * p.n + w.col() : -1;
            zv[u] = at[u] >= 0 ? ptx::ld_stream(static_cast<const uint16_t *>(p.z) + at[u]) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        f32x2 f[4];
        unpack8<DT>(zv[u], f);
        float big = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) big = max_abs(big, f[e]);
        uint32_t top = __float_as_uint(big);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t ex = ckpt_exponent(top), id = id0 + u * (CKPT_T / 4);
        if (at[u] >= 0) {
            *reinterpret_cast<uint2 *>(p.codes + at[u]) = codes8<NORM_I8_ROWS>(f, ckpt_inverse(ex));
            if (p.h != nullptr) {
                ckpt_act8<EPI>(f);
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.h) + at[u]) = pack8<DT>(f);
            }
        }
        if ((threadIdx.x & 3) == 0 && id < p.total) p.exps[id] = (uint8_t)ex;
    }
}

template <int DT, int EPI, int U>
__global__ void __launch_bounds__(CKPT_T) ckpt_load_kernel(const CkptParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    uint2 q[U];
    uint32_t ex[U];
    int64_t at[U];
    CkptWalk w(p, U);
#pragma unroll
    for (int u = 0; u < U; ++u, w.next(p)) {
        at[u] = w.id < p.total && w.col() < p.n ? (int64_t)w.row * p.n + w.col() : -1;
        q[u] = make_uint2(0u, 0u);
        ex[u] = 7u;
        if (at[u] >= 0) {
            q[u] = __ldg(reinterpret_cast<const uint2 *>(p.codes + at[u]));
            ex[u] = __ldg(p.exps + w.id);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        f32x2 f[4];
        ckpt_decode8(q[u], ckpt_step(ex[u]), f);
        ckpt_act8<EPI>(f);
        if constexpr (EPI != EPI_TANH) ckpt_draw_back8<DT>(f, ex[u]);
        if (at[u] >= 0) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.h) + at[u]) = pack8<DT>(f);
    }
}

}  // namespace gemm_epi
