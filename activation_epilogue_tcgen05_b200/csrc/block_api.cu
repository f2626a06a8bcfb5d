// block_api.cu -- C ABI of the operators around the MLP's products: the norm before them and its
// backward (rmsnorm.cuh), and the backward of their epilogue (dact.cuh).  Argument checks come
// before the device is looked at; nothing is allocated here.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "../../include/gemm_epi.h"
#include "dact.cuh"
#include "kernels.h"
#include "rmsnorm.cuh"

using namespace gemm_epi;

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// GEMM_EPI_OK on a compute-capability 10.0 device (looked up once a device).
int check_device() {
    static std::atomic<signed char> known[64];      // 0 not looked up, 1 sm_100, -1 another
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
        cudaGetLastError();
        return GEMM_EPI_ERR_NO_DEVICE;
    }
    signed char k = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (k == 0) {
        int major = 0, minor = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        k = major == 10 && minor == 0 ? 1 : -1;
        if (dev < 64) known[dev].store(k, std::memory_order_relaxed);
    }
    return k == 1 ? GEMM_EPI_OK : GEMM_EPI_ERR_NO_DEVICE;
}

bool pdl_enabled() {
    const char *e = getenv("GEMM_EPI_PDL");
    return !(e && e[0] == '0');
}

int status(cudaError_t e) {
    if (e != cudaSuccess && getenv("GEMM_EPI_LOG")) fprintf(stderr, "gemm_epi launch: %s (%d)\n", cudaGetErrorString(e), (int)e);
    return e == cudaSuccess ? GEMM_EPI_OK : GEMM_EPI_ERR_CUDA;
}

// sizes, type and eps of a norm; d_multiple: what d has to be a multiple of
int check_norm(int64_t m, int64_t d, int dtype, float eps, int64_t d_multiple) {
    if (m <= 0 || d <= 0 || m > 0x7fffffffll || d > 0x7fffffffll) return GEMM_EPI_ERR_ARG;
    if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return GEMM_EPI_ERR_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return GEMM_EPI_ERR_ARG;
    if (d % d_multiple != 0) return GEMM_EPI_ERR_ALIGN;
    if (d > NORM_MAX_D) return GEMM_EPI_ERR_UNSUPPORTED;
    return GEMM_EPI_OK;
}

}  // namespace

extern "C" {

int gemm_epi_rmsnorm(int64_t m, int64_t d, int dtype, int out_mode, float eps, const void *X, const void *R,
                     const void *gamma, void *S, void *Y, float *d_scale, float *d_amax, void *stream) {
    if (out_mode < GEMM_EPI_NORM_SAME || out_mode > GEMM_EPI_NORM_E4M3_ROWS) return GEMM_EPI_ERR_ARG;
    int rc = check_norm(m, d, dtype, eps, out_mode == GEMM_EPI_NORM_SAME ? 8 : 16);
    if (rc != GEMM_EPI_OK) return rc;
    if (!X || !gamma || !Y || (out_mode != GEMM_EPI_NORM_SAME && !d_scale)) return GEMM_EPI_ERR_NULL;
    if (!R && S) return GEMM_EPI_ERR_ARG;                       // the sum is X itself
    if (S == Y) return GEMM_EPI_ERR_ARG;
    if (out_mode != GEMM_EPI_NORM_SAME && (Y == X || Y == R)) return GEMM_EPI_ERR_ARG;   // rows of another pitch
    if (!aligned(X, 16) || !aligned(R, 16) || !aligned(gamma, 16) || !aligned(S, 16) || !aligned(Y, 16) ||
        !aligned(d_scale, 4) || !aligned(d_amax, 4))
        return GEMM_EPI_ERR_ALIGN;
    rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    NormParams p{};
    p.m = m;
    p.d = (int)d;
    p.eps = eps;
    p.inv_d = 1.0f / (float)d;
    p.x = X;
    p.r = R;
    p.gamma = gamma;
    p.s = S;
    p.y = Y;
    p.scale = d_scale;
    p.amax = out_mode == GEMM_EPI_NORM_E4M3 ? reinterpret_cast<unsigned int *>(d_amax) : nullptr;
    // the amax word is this call's maximum: start it at 0 (the kernel max-reduces into it)
    const bool pdl = pdl_enabled();
    if (p.amax && (rc = status(launch_zero_word(p.amax, pdl, s))) != GEMM_EPI_OK) return rc;
    return status(launch_rmsnorm(dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16, out_mode, p, pdl, s));
}

int64_t gemm_epi_rmsnorm_workspace_bytes(int64_t m, int64_t d) {
    if (m <= 0 || d <= 0 || d > NORM_MAX_D || d % 8 != 0 || m > 0x7fffffffll) return 0;
    return norm_bwd_parts(m, d) * d * (int64_t)sizeof(float);
}

int gemm_epi_rmsnorm_bwd(int64_t m, int64_t d, int dtype, float eps, const void *dY, const void *S, const void *gamma,
                         const void *dS, void *dX, void *dgamma, void *workspace, void *stream) {
    int rc = check_norm(m, d, dtype, eps, 8);
    if (rc != GEMM_EPI_OK) return rc;
    const int64_t parts = dgamma ? norm_bwd_parts(m, d) : 0;
    if (!dY || !S || !gamma || !dX || (parts > 0 && !workspace)) return GEMM_EPI_ERR_NULL;
    if (!aligned(dY, 16) || !aligned(S, 16) || !aligned(gamma, 16) || !aligned(dS, 16) || !aligned(dX, 16) ||
        !aligned(dgamma, 16) || !aligned(workspace, 16))
        return GEMM_EPI_ERR_ALIGN;
    rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int dt = dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16;
    NormBwdParams p{};
    p.m = m;
    p.d = (int)d;
    p.eps = eps;
    p.inv_d = 1.0f / (float)d;
    p.dy = dY;
    p.s = S;
    p.gamma = gamma;
    p.ds = dS;
    p.dx = dX;
    p.partial = parts > 0 ? static_cast<float *>(workspace) : nullptr;
    p.dgamma = parts > 0 ? nullptr : dgamma;
    const bool pdl = pdl_enabled();
    rc = status(launch_rmsnorm_bwd(dt, p, pdl, s));
    if (rc != GEMM_EPI_OK || parts == 0) return rc;
    return status(launch_add_parts(dt, p.partial, parts, d, dgamma, pdl, s));
}

int64_t gemm_epi_dact_workspace_bytes(int64_t m, int64_t n, int bias_axis) {
    if (m <= 0 || n <= 0 || m > 0x7fffffffll || n > 0x7fffffffll) return 0;
    if (n % 8 != 0) return 0;
    if (bias_axis == GEMM_EPI_BIAS_ROW && dact_by_rows(m, n)) return 0;
    if (bias_axis == GEMM_EPI_BIAS_ROW) return (n + DACT_COLS - 1) / DACT_COLS * m * (int64_t)sizeof(float);
    if (bias_axis != GEMM_EPI_BIAS_COL) return 0;
    const int64_t rows = std::min(dact_rows(m, n, true), dact_rows(m, n, false));      // whatever the epilogue
    return rows >= m ? 0 : (m + rows - 1) / rows * n * (int64_t)sizeof(float);
}

int gemm_epi_dact(int64_t m, int64_t n, int dtype, int epilogue, int bias_axis, const void *dD, const void *Z,
                  const uint32_t *aux, void *dZ, void *dbias, void *workspace, void *stream) {
    if (m <= 0 || n <= 0 || m > 0x7fffffffll || n > 0x7fffffffll) return GEMM_EPI_ERR_ARG;
    if (dtype < GEMM_EPI_F16 || dtype > GEMM_EPI_E4M3) return GEMM_EPI_ERR_ARG;
    if (bias_axis != GEMM_EPI_BIAS_ROW && bias_axis != GEMM_EPI_BIAS_COL) return GEMM_EPI_ERR_ARG;
    int act;
    switch (epilogue) {
    case GEMM_EPI_NONE: case GEMM_EPI_BIAS: act = DACT_NONE; break;
    case GEMM_EPI_RELU: case GEMM_EPI_RELU_BIAS: act = DACT_RELU; break;
    case GEMM_EPI_RELU_AUX: case GEMM_EPI_RELU_AUX_BIAS: act = DACT_RELU_MASK; break;
    case GEMM_EPI_GELU: case GEMM_EPI_GELU_BIAS: act = DACT_GELU; break;
    case GEMM_EPI_TANH: case GEMM_EPI_TANH_BIAS: act = DACT_TANH; break;
    default: return GEMM_EPI_ERR_ARG;
    }
    if (n % 8 != 0) return GEMM_EPI_ERR_ALIGN;
    const bool mask = act == DACT_RELU_MASK;
    if (!dD || (mask && !aux) || (!mask && act != DACT_NONE && !Z)) return GEMM_EPI_ERR_NULL;
    if (act == DACT_NONE ? !dbias : !dZ) return GEMM_EPI_ERR_NULL;
    // the sums end in a block each: rows whole in a block, or all rows in one run
    const int64_t rows = dact_rows(m, n, dact_reads_z(act));
    const bool at_once = dbias && (bias_axis == GEMM_EPI_BIAS_ROW ? dact_by_rows(m, n) : rows >= m);
    if (dbias && !at_once && !workspace) return GEMM_EPI_ERR_NULL;
    if (act == DACT_NONE && dZ) return GEMM_EPI_ERR_ARG;          // dZ is dD itself
    if (!aligned(dD, 16) || (act != DACT_NONE && !mask && !aligned(Z, 16)) || (mask && !aligned(aux, 16)) ||
        !aligned(dZ, 16) || !aligned(dbias, 16) || !aligned(workspace, 16))
        return GEMM_EPI_ERR_ALIGN;
    int rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int dt = dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16;      // e4m3 operands have bf16 outputs
    const int axis = bias_axis == GEMM_EPI_BIAS_COL ? AXIS_COL : AXIS_ROW;
    DactParams p{};
    p.m = m;
    p.n = (int)n;
    p.rows = rows;
    p.dd = dD;
    p.z = Z;
    p.aux = reinterpret_cast<const uint8_t *>(aux);
    p.aux_pitch = gemm_epi_aux_pitch_bytes(n);
    p.dz = dZ;
    p.partial = dbias && !at_once ? static_cast<float *>(workspace) : nullptr;
    p.dbias = at_once ? dbias : nullptr;
    const bool pdl = pdl_enabled();
    rc = status(launch_dact(dt, act, axis, p, pdl, s));
    if (rc != GEMM_EPI_OK || !p.partial) return rc;
    const int64_t parts = axis == AXIS_COL ? (m + p.rows - 1) / p.rows : (n + DACT_COLS - 1) / DACT_COLS;
    const int64_t len = axis == AXIS_COL ? n : m;
    return status(len % 8 == 0 ? launch_add_parts(dt, p.partial, parts, len, dbias, pdl, s)
                               : launch_sum_parts_f32(dt, p.partial, parts, len, dbias, pdl, s));      // ROW, odd m
}

}  // extern "C"
