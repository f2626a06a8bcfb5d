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
//
// z may also come from its checkpoint in 8 bits (CK; ckpt.cuh): codes through the ring, 8 bytes a lane, one exponent for 32
// columns a batch ahead in registers; and act(z) may be written beside dZ, from the slope's own terms.
#pragma once
#include <cstdint>

#include "ckpt.cuh"
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
    const int8_t *codes;     // CK: z's checkpoint in place of z
    const uint8_t *exps;     // [m][ckpt_groups(n)]
    void *h;                 // CK: act(z) in the 16-bit type, or NULL
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
// Phi's own tail comes out on the way, and with it the value: GELU(x) = max(x, 0) - u (1 - Phi(u)) (val; for finite x, FINITE: which need no cut).
template <bool FINITE = false>
__device__ __forceinline__ f32x2 gelu_slope(float x0, float x1, f32x2 *val = nullptr) {
    constexpr float c = 0.84932180028801907f;                                 // sqrt(log2(e) / 2): e = 2^-(c u)^2
    const f32x2 u = pair(fabsf(x0), fabsf(x1));
    const f32x2 v = mul2(FINITE ? u : pair(min_nan(fabsf(x0), 16.0f), min_nan(fabsf(x1), 16.0f)), both(c));
    const float2 den = split(add2(v, both(2.498f))), q = split(mul2(v, v));
    const f32x2 t = pair(rcp_approx(den.x), rcp_approx(den.y));
    f32x2 h = fma2(t, both(20.0101986f), both(-24.893486f));
    h = fma2(t, h, both(0.832031548f));
    h = fma2(t, h, both(-2.2361939f));
    h = fma2(t, h, both(-0.653034389f));
    h = mul2(t, h);                                                           // -2 exp(u^2 / 2) (1 - Phi(u))
    const f32x2 w = fma2(v, both(2.0f * 0.39894228040143268f / c), h);        // -2 w(u)
    const f32x2 e = pair(ex2_approx(-q.x), ex2_approx(-q.y));
    const f32x2 left = mul2(e, w);
    if (val != nullptr)
        *val = fma2(mul2(u, both(0.5f)), mul2(e, h), pair(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f)));
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

// act'(z) of two neighbouring elements; val: act(z) as well, if wanted.
template <int ACT, bool FINITE>
__device__ __forceinline__ f32x2 slope(f32x2 z, f32x2 *val = nullptr) {
    const float2 x = split(z);
    if constexpr (ACT == DACT_GELU) return gelu_slope<FINITE>(x.x, x.y, val);
    if (val != nullptr) *val = tanh2(x.x, x.y);
    return tanh_slope(x.x, x.y);
}

// d *= act'(z) for a lane's eight elements (bits: their mask); VAL: z becomes act(z).  CK: z is finite or, in a group that save found
// not to be, NaN throughout, and d becomes NaN with it: GELU's and tanh's slopes are NaN there, and ReLU's, a comparison,
// takes the place of its 0 from the first element.
template <int ACT, bool CK, bool VAL>
__device__ __forceinline__ void through_act(f32x2 (&d)[4], f32x2 (&z)[4], uint32_t bits) {
    float none = 0.0f;
    if constexpr (CK && ACT == DACT_RELU) {
        const float first = split(z[0]).x;
        if (first != first) none = first;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (ACT == DACT_RELU_MASK) {
            const float2 f = split(d[e]);
            d[e] = pair(((bits >> 2 * e) & 1u) ? f.x : 0.0f, ((bits >> (2 * e + 1)) & 1u) ? f.y : 0.0f);
        } else if constexpr (ACT == DACT_RELU) {
            const float2 f = split(d[e]), x = split(z[e]);
            d[e] = pair(x.x > 0.0f ? f.x : none, x.y > 0.0f ? f.y : none);
            if constexpr (VAL) z[e] = pair(x.x < 0.0f ? 0.0f : x.x, x.y < 0.0f ? 0.0f : x.y);
        } else if constexpr (ACT != DACT_NONE) {
            f32x2 val;
            d[e] = mul2(d[e], slope<ACT, CK>(z[e], VAL ? &val : nullptr));
            if constexpr (VAL) z[e] = val;
        }
    }
}

// Sum of a lane's eight elements, neighbours first.
__device__ __forceinline__ float sum8(const f32x2 (&d)[4]) {
    const float2 a = split(d[0]), b = split(d[1]), c = split(d[2]), e = split(d[3]);
    return ((a.x + a.y) + (b.x + b.y)) + ((c.x + c.y) + (e.x + e.y));
}

// With z to read, rows go through a ring of batches in shared memory, each thread copying its own vectors
// (cp.async, as the norm's backward does): the next batch is on its way while the slopes of one are
// worked out (8192 x 14336 GELU 114 us, loaded where it is used 134).  Without z there is little to work
// out, and a batch is loaded into registers by four blocks an SM instead of three (bias alone 38.6 us,
// through a ring 40.6; 1023 x 4104 from the mask 5.4 us against 7.0; f16 along rows in strips from the mask spills 20 bytes a thread).
constexpr int DACT_U = 4;                             // rows of a warp in a batch (CK: their exponents share a word)
constexpr bool dact_reads_z(int act) { return act != DACT_NONE && act != DACT_RELU_MASK; }
// Where a slope is computed, two rows of a batch are worked out at a time: with all four interleaved the constants no longer
// fit the 80 registers that three blocks an SM leave (8192 x 14336 GELU 120 us, two at a time 112).
constexpr bool dact_computes(int act) { return act == DACT_GELU || act == DACT_TANH; }
// Blocks an SM.  From a checkpoint two, at up to 128 registers: a batch's four rows are worked out together (rows whole in a
// block and act(z) as well: two by two), with the codes taken apart and act(z) on top of the slope's constants (8192 x 14336
// GELU with act(z) 136 us; three blocks, two rows at a time 157, one at a time 140; without act(z) 107 and 109).
constexpr int dact_blocks(int act, bool ck) { return ck ? 2 : dact_reads_z(act) ? 3 : 4; }
constexpr int DACT_RING = 2;
constexpr int dact_smem(bool ck, int u = DACT_U) { return DACT_RING * u * 32 * DACT_WARPS * (ck ? 24 : 32); }

// What a thread has of one row of a stage in the ring: [DACT_RING][U][T] of dD, then as many of z or of its codes.  Where there is
// no row (or column) left the thread puts zeros there, so that nothing that is read has to be asked about: 0 adds nothing
// to a sum.
template <bool CK, int U = DACT_U>
struct DactRing {
    using Zv = std::conditional_t<CK, uint2, uint4>;
    using Zg = std::conditional_t<CK, int8_t, uint16_t>;
    static constexpr int T = 32 * DACT_WARPS, N = DACT_RING * U * T;
    static __device__ __forceinline__ uint4 *dd(uint4 *ring, int stage, int u) { return ring + (stage * U + u) * T + threadIdx.x; }
    static __device__ __forceinline__ Zv *z(uint4 *ring, int stage, int u) {
        return reinterpret_cast<Zv *>(ring + N) + (stage * U + u) * T + threadIdx.x;
    }
    static __device__ __forceinline__ void fetch(uint4 *ring, int stage, int u, bool ok, const uint16_t *from, const Zg *zfrom) {
        if (ok) {
            ptx::cp_async_16(dd(ring, stage, u), from);
            if constexpr (CK) ptx::cp_async_8(z(ring, stage, u), zfrom);
            else ptx::cp_async_16(z(ring, stage, u), zfrom);
        } else {
            *dd(ring, stage, u) = make_uint4(0u, 0u, 0u, 0u);
            *z(ring, stage, u) = Zv{};
        }
    }
    // z as values; ex: its exponent (CK)
    template <int DT>
    static __device__ __forceinline__ void values(uint4 *ring, int stage, int u, uint32_t ex, f32x2 (&f)[4]) {
        if constexpr (CK) ckpt_decode8(*z(ring, stage, u), ckpt_step(ex), f);
        else unpack8<DT>(*z(ring, stage, u), f);
    }
};

template <int DT, int ACT, int AXIS, bool CK = false, bool VAL = false>
__global__ void __launch_bounds__(32 * DACT_WARPS, dact_blocks(ACT, CK)) dact_kernel(const DactParams p) {
    constexpr int U = DACT_U;
    constexpr bool Z = dact_reads_z(ACT), SLOPE = dact_computes(ACT);
    static_assert(Z || !CK, "a checkpoint is one of z");
    using Ring = DactRing<CK>;
    extern __shared__ uint4 ring[];                   // Z: Ring
    __shared__ float4 sums[AXIS == AXIS_COL ? 64 * DACT_WARPS : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * DACT_COLS + 8 * lane;
    const bool col_ok = col < p.n;                    // n is a multiple of 8
    const int64_t r0 = (int64_t)blockIdx.y * p.rows + warp;
    // the warp's rows: every DACT_WARPS-th of the run's; `at` is where this lane's values of one lie
    const int rows = (int)min(p.rows, p.m - (int64_t)blockIdx.y * p.rows);
    constexpr int step = U * DACT_WARPS;
    const int64_t pitch = (int64_t)DACT_WARPS * p.n;
    int64_t at = r0 * p.n + col;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint16_t *dd = static_cast<const uint16_t *>(p.dd);
    auto fetch = [&](int r, int64_t at, int stage) {
        const typename Ring::Zg *z = reinterpret_cast<const typename Ring::Zg *>(CK ? static_cast<const void *>(p.codes) : p.z);
#pragma unroll
        for (int u = 0; u < U; ++u, at += pitch) Ring::fetch(ring, stage, u, r + u * DACT_WARPS < rows && col_ok, dd + at, z + at);
        ptx::cp_async_commit();
    };
    // CK: the coming batch's exponents
    uint32_t next[U];
    const int groups = ckpt_groups(p.n);
    const uint8_t *ex_at = CK ? p.exps + r0 * groups + col / CKPT_GROUP : nullptr;
    auto exponents = [&](int r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next[u] = 7u;
            if (r + u * DACT_WARPS < rows && col_ok) next[u] = __ldg(ex_at + (int64_t)(u * DACT_WARPS) * groups);
        }
        ex_at += (int64_t)step * groups;
    };
    f32x2 acc[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
    int r = warp;
    if constexpr (Z) {
#pragma unroll
        for (int i = 0; i < DACT_RING; ++i) fetch(r + i * step, at + i * U * pitch, i);
        if constexpr (CK) exponents(r);
    }
    int stage = 0;
    for (; r < rows; r += step, at += U * pitch) {
        uint4 dv[U];
        uint32_t bits[U], ex = 0u;                    // the mask's; CK: the rows' exponents, a byte each
        if constexpr (Z) {
            if constexpr (CK) {
                ex = next[0] | next[1] << 8 | next[2] << 16 | next[3] << 24;
                exponents(r + step);
            }
            ptx::cp_async_wait<DACT_RING - 1>();
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                dv[u] = make_uint4(0u, 0u, 0u, 0u);
                bits[u] = 0u;
                if (r + u * DACT_WARPS < rows && col_ok) {
                    dv[u] = ptx::ld_stream(dd + at + u * pitch);
                    if constexpr (ACT == DACT_RELU_MASK) bits[u] = __ldg(p.aux + (r0 - warp + r + u * DACT_WARPS) * p.aux_pitch + col / 8);
                }
            }
        }
        int64_t to = at;
        constexpr int AT_ONCE = SLOPE && !CK ? 2 : U;
#pragma unroll AT_ONCE
        for (int u = 0; u < U; ++u, to += pitch) {
            const bool row_ok = r + u * DACT_WARPS < rows;
            f32x2 d[4], z[4];
            if constexpr (Z) {
                unpack8<DT>(*Ring::dd(ring, stage, u), d);
                Ring::template values<DT>(ring, stage, u, ex >> 8 * u & 255u, z);
            } else {
                unpack8<DT>(dv[u], d);
            }
            through_act<ACT, CK, VAL>(d, z, bits[u]);
            if constexpr (VAL && ACT != DACT_TANH) ckpt_draw_back8<DT>(z, ex >> 8 * u & 255u);
            if (row_ok && col_ok) {
                if constexpr (ACT != DACT_NONE) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dz) + to) = pack8<DT>(d);
                if constexpr (VAL) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.h) + to) = pack8<DT>(z);
            }
            if constexpr (AXIS == AXIS_COL) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = add2(acc[e], d[e]);
            } else if (p.partial != nullptr) {
                float s = sum8(d);
#pragma unroll
                for (int sh = 16; sh >= 1; sh >>= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
                if (lane == 0 && row_ok) p.partial[(int64_t)blockIdx.x * p.m + (r0 - warp + r + u * DACT_WARPS)] = s;
            }
        }
        if constexpr (Z) {
            fetch(r + DACT_RING * step, at + DACT_RING * U * pitch, stage);
            if (++stage == DACT_RING) stage = 0;
        }
    }
    if constexpr (Z) ptx::cp_async_wait<0>();
    if constexpr (AXIS == AXIS_COL) {
        if (p.partial == nullptr && p.dbias == nullptr) return;
        // the warps' sums, in order: [warp][half of a lane's 8][lane]
        sums[(2 * warp) * 32 + lane] = quad(acc[0], acc[1]);
        sums[(2 * warp + 1) * 32 + lane] = quad(acc[2], acc[3]);
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

// The bias along the rows: a block takes U rows whole, its warps side by side on 2048 columns at a
// time, so that a row's sum ends in the block and dbias is written at once: one launch, no scratch, and one
// butterfly a row instead of one every 256 columns (8192 x 14336 ReLU 106 us against 115, 1023 x 4104 from the
// mask 6.7 us a call from Python against 11.0).  The same ring, along the columns.
template <int DT, int ACT, bool CK = false, bool VAL = false, int U = DACT_U>
__global__ void __launch_bounds__(32 * DACT_WARPS, U == DACT_U ? dact_blocks(ACT, CK) : 3) dact_rows_kernel(const DactParams p) {
    constexpr int PASS = DACT_WARPS * DACT_COLS;
    constexpr bool Z = dact_reads_z(ACT), SLOPE = dact_computes(ACT);
    static_assert(U % 2 == 0 && U <= 4, "rows are worked out two at a time; their exponents share a word");
    static_assert(Z || !CK, "a checkpoint is one of z");
    using Ring = DactRing<CK, U>;
    extern __shared__ uint4 ring[];                   // Z: Ring
    __shared__ float sums[DACT_WARPS][U];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * U;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint16_t *dd = static_cast<const uint16_t *>(p.dd) + r0 * p.n;
    const typename Ring::Zg *zz = reinterpret_cast<const typename Ring::Zg *>(CK ? static_cast<const void *>(p.codes) : p.z) + (Z ? r0 * p.n : 0);
    uint16_t *dz = static_cast<uint16_t *>(p.dz) + r0 * p.n;
    uint16_t *hh = VAL ? static_cast<uint16_t *>(p.h) + r0 * p.n : nullptr;
    const int rows = (int)min((int64_t)U, p.m - r0);
    auto fetch = [&](int64_t col, int stage) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            Ring::fetch(ring, stage, u, u < rows && col < p.n, dd + (int64_t)u * p.n + col, zz + (int64_t)u * p.n + col);
        ptx::cp_async_commit();
    };
    const int groups = ckpt_groups(p.n);
    uint32_t next[U];                                 // CK: the coming pass's exponents
    auto exponents = [&](int64_t col) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next[u] = 7u;
            if (u < rows && col < p.n) next[u] = __ldg(p.exps + (r0 + u) * groups + col / CKPT_GROUP);
        }
    };
    float acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u] = 0.0f;
    int64_t col = 8 * threadIdx.x;                    // (n may be within a pass of 2^31)
    if constexpr (Z) {
#pragma unroll
        for (int i = 0; i < DACT_RING; ++i) fetch(col + i * PASS, i);
        if constexpr (CK) exponents(col);
    }
    int stage = 0;
    for (; col < p.n; col += PASS) {
        uint4 dv[U];
        uint32_t bits[U], ex = 0u;                    // the mask's; CK: the rows' exponents, a byte each
        if constexpr (Z) {
            if constexpr (CK) {
#pragma unroll
                for (int u = 0; u < U; ++u) ex |= next[u] << 8 * u;
                exponents(col + PASS);
            }
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
        constexpr int AT_ONCE = SLOPE && (!CK || VAL) ? 1 : U / 2;
#pragma unroll AT_ONCE
        for (int u0 = 0; u0 < U; u0 += 2) {
            float sum[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int u = u0 + k;
                f32x2 d[4], z[4];
                if constexpr (Z) {
                    unpack8<DT>(*Ring::dd(ring, stage, u), d);
                    Ring::template values<DT>(ring, stage, u, ex >> 8 * u & 255u, z);
                } else {
                    unpack8<DT>(dv[u], d);
                }
                through_act<ACT, CK, VAL>(d, z, bits[u]);
                if constexpr (VAL && ACT != DACT_TANH) ckpt_draw_back8<DT>(z, ex >> 8 * u & 255u);
                if (u < rows) {
                    if constexpr (ACT != DACT_NONE) *reinterpret_cast<uint4 *>(dz + (int64_t)u * p.n + col) = pack8<DT>(d);
                    if constexpr (VAL) *reinterpret_cast<uint4 *>(hh + (int64_t)u * p.n + col) = pack8<DT>(z);
                }
                sum[k] = acc[k] + sum8(d);
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

// The bias along narrow rows, many of them, from a checkpoint: a warp takes rows whole, strip of 256 columns by strip, so that a
// row's sum ends in the warp and no thread is without columns but for the last strip's (65536 x 1024 GELU 75 us, in blocks of
// whole rows 127).
template <int DT, int ACT, bool VAL>
__global__ void __launch_bounds__(32 * DACT_WARPS, dact_blocks(ACT, true)) dact_narrow_kernel(const DactParams p) {
    constexpr int U = DACT_U;
    using Ring = DactRing<true>;
    extern __shared__ uint4 ring[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int strips = (p.n + DACT_COLS - 1) / DACT_COLS, groups = ckpt_groups(p.n);
    const int64_t step = (int64_t)gridDim.x * DACT_WARPS;
    // a strip of a row, and the warp's next one
    struct Item {
        int64_t row;
        int strip;
    };
    auto next = [&](Item &i) {
        if (++i.strip == strips) {
            i.strip = 0;
            i.row += step;
        }
    };
    Item now{(int64_t)blockIdx.x * DACT_WARPS + warp, 0}, ahead = now;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    uint32_t ex[U];                                   // exponents of the batch that was asked for last
    auto fetch = [&](int stage) {
#pragma unroll
        for (int u = 0; u < U; ++u, next(ahead)) {
            const int col = ahead.strip * DACT_COLS + 8 * lane;
            const bool ok = ahead.row < p.m && col < p.n;
            const int64_t at = ahead.row * p.n + col;
            Ring::fetch(ring, stage, u, ok, static_cast<const uint16_t *>(p.dd) + at, p.codes + at);
            ex[u] = ok ? __ldg(p.exps + ahead.row * groups + col / CKPT_GROUP) : 7u;
        }
        ptx::cp_async_commit();
    };
    auto word = [&]() { return ex[0] | ex[1] << 8 | ex[2] << 16 | ex[3] << 24; };
    fetch(0);
    uint32_t coming = word();
    fetch(1);
    static_assert(DACT_RING == 2, "two batches ahead");
    float sum = 0.0f;
    for (int stage = 0; now.row < p.m; stage ^= 1) {
        const uint32_t cur = coming;
        coming = word();
        ptx::cp_async_wait<DACT_RING - 1>();
#pragma unroll
        for (int u = 0; u < U; ++u, next(now)) {
            const int col = now.strip * DACT_COLS + 8 * lane;
            f32x2 d[4], z[4];
            unpack8<DT>(*Ring::dd(ring, stage, u), d);
            Ring::template values<DT>(ring, stage, u, cur >> 8 * u & 255u, z);
            through_act<ACT, true, VAL>(d, z, 0u);
            if constexpr (VAL && ACT != DACT_TANH) ckpt_draw_back8<DT>(z, cur >> 8 * u & 255u);
            if (now.row < p.m && col < p.n) {
                const int64_t at = now.row * p.n + col;
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.dz) + at) = pack8<DT>(d);
                if constexpr (VAL) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.h) + at) = pack8<DT>(z);
            }
            sum += sum8(d);
            if (now.strip == strips - 1) {
#pragma unroll
                for (int sh = 16; sh >= 1; sh >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
                if (lane == 0 && now.row < p.m) static_cast<uint16_t *>(p.dbias)[now.row] = (uint16_t)OutT<DT>::pack(sum, 0.0f);
                sum = 0.0f;
            }
        }
        fetch(stage);
    }
    ptx::cp_async_wait<0>();
}

}  // namespace gemm_epi
