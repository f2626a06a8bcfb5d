// block_api.cu -- C ABI of the operators around the MLP's products: the norms before them and their
// backward (rmsnorm.cuh, layernorm.cuh), rows quantised for them, the backward of their epilogue (dact.cuh) and the
// 8-bit checkpoints it may read (ckpt.cuh).  Argument checks come before the device is looked at; nothing is allocated here.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "../../include/gemm_epi.h"
#include "ckpt.cuh"
#include "dact.cuh"
#include "kernels.h"
#include "layernorm.cuh"
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

// The arguments that both norms share, checked and laid out (beta: the layer norm's, else NULL).
int norm_params(int64_t m, int64_t d, int dtype, int out_mode, float eps, const void *X, const void *R, const void *gamma,
                const void *beta, void *S, void *Y, float *d_scale, float *d_amax, NormParams *p) {
    const bool by_rows = out_mode == GEMM_EPI_NORM_E4M3_ROWS || out_mode == GEMM_EPI_NORM_I8_ROWS;
    if (out_mode != GEMM_EPI_NORM_SAME && out_mode != GEMM_EPI_NORM_E4M3 && !by_rows) return GEMM_EPI_ERR_ARG;
    int rc = check_norm(m, d, dtype, eps, out_mode == GEMM_EPI_NORM_SAME ? 8 : 16);
    if (rc != GEMM_EPI_OK) return rc;
    if (!X || !gamma || !Y || (out_mode != GEMM_EPI_NORM_SAME && !d_scale)) return GEMM_EPI_ERR_NULL;
    if (!R && S) return GEMM_EPI_ERR_ARG;                       // the sum is X itself
    if (S == Y) return GEMM_EPI_ERR_ARG;
    if (out_mode != GEMM_EPI_NORM_SAME && (Y == X || Y == R)) return GEMM_EPI_ERR_ARG;   // rows of another pitch
    if (!aligned(X, 16) || !aligned(R, 16) || !aligned(gamma, 16) || !aligned(beta, 16) || !aligned(S, 16) || !aligned(Y, 16) ||
        !aligned(d_scale, 4) || !aligned(d_amax, 4))
        return GEMM_EPI_ERR_ALIGN;
    rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    p->m = m;
    p->d = (int)d;
    p->eps = eps;
    p->inv_d = 1.0f / (float)d;
    p->x = X;
    p->r = R;
    p->gamma = gamma;
    p->s = S;
    p->y = Y;
    p->scale = d_scale;
    p->amax = out_mode == GEMM_EPI_NORM_E4M3 ? reinterpret_cast<unsigned int *>(d_amax) : nullptr;
    return GEMM_EPI_OK;
}

// The activation of a backward call, or -1 for an epilogue it does not know.
int dact_of_epilogue(int epilogue) {
    switch (epilogue) {
    case GEMM_EPI_NONE: case GEMM_EPI_BIAS: return DACT_NONE;
    case GEMM_EPI_RELU: case GEMM_EPI_RELU_BIAS: return DACT_RELU;
    case GEMM_EPI_RELU_AUX: case GEMM_EPI_RELU_AUX_BIAS: return DACT_RELU_MASK;
    case GEMM_EPI_GELU: case GEMM_EPI_GELU_BIAS: return DACT_GELU;
    case GEMM_EPI_TANH: case GEMM_EPI_TANH_BIAS: return DACT_TANH;
    default: return -1;
    }
}

// The forward activation (EPI_*) of a checkpoint's epilogue, or -1.
int act_of_epilogue(int epilogue) {
    switch (dact_of_epilogue(epilogue)) {
    case DACT_NONE: return EPI_NONE;
    case DACT_RELU: case DACT_RELU_MASK: return EPI_RELU;
    case DACT_GELU: return EPI_GELU;
    case DACT_TANH: return EPI_TANH;
    default: return -1;
    }
}

// Sizes, type and epilogue of a checkpoint.
int check_ckpt(int64_t m, int64_t n, int dtype, int epilogue) {
    if (m <= 0 || n <= 0 || m > 0x7fffffffll || n > 0x7fffffffll) return GEMM_EPI_ERR_ARG;
    if (dtype < GEMM_EPI_F16 || dtype > GEMM_EPI_E4M3) return GEMM_EPI_ERR_ARG;
    if (act_of_epilogue(epilogue) < 0) return GEMM_EPI_ERR_ARG;
    if (n % 8 != 0) return GEMM_EPI_ERR_ALIGN;
    // (groups are counted in 32 bits, and a block's run past the last one has to fit)
    if (m * ckpt_groups(n) > 0xFFFFFF00ll) return GEMM_EPI_ERR_UNSUPPORTED;
    return GEMM_EPI_OK;
}

int run_ckpt(bool save, int64_t m, int64_t n, int dtype, int epilogue, const void *Z, void *H, int8_t *codes, uint8_t *exps,
             void *stream) {
    CkptParams p{};
    p.n = (int)n;
    p.groups = (uint32_t)ckpt_groups(n);
    p.total = (uint32_t)(m * ckpt_groups(n));
    p.z = Z;
    p.h = H;
    p.codes = codes;
    p.exps = exps;
    return status(launch_ckpt(dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16, save, act_of_epilogue(epilogue), p, pdl_enabled(),
                              static_cast<cudaStream_t>(stream)));
}

// Whether dbias's sums go through the workspace.  They do not where they end in a block each: rows whole in a block, or all
// rows in one run.
bool dact_needs_workspace(int64_t m, int64_t n, int blocks, int bias_axis) {
    return !(bias_axis == GEMM_EPI_BIAS_ROW ? dact_by_rows(m, n) : dact_rows(m, n, blocks) >= m);
}

// Launches of an epilogue's backward: the strips or whole rows, then what adds their sums up.
int run_dact(DactParams &p, int64_t m, int64_t n, int dtype, int act, int bias_axis, bool ckpt, void *dbias, void *workspace,
             void *stream) {
    const int blocks = dact_blocks(act, ckpt);
    const bool at_once = dbias && !dact_needs_workspace(m, n, blocks, bias_axis);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int dt = dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16;      // e4m3 operands have bf16 outputs
    const int axis = bias_axis == GEMM_EPI_BIAS_COL ? AXIS_COL : AXIS_ROW;
    p.m = m;
    p.n = (int)n;
    p.rows = dact_rows(m, n, blocks);
    p.partial = dbias && !at_once ? static_cast<float *>(workspace) : nullptr;
    p.dbias = at_once ? dbias : nullptr;
    const bool pdl = pdl_enabled();
    const int rc = status(ckpt ? launch_dact_ckpt(dt, act, axis, p, pdl, s) : launch_dact(dt, act, axis, p, pdl, s));
    if (rc != GEMM_EPI_OK || !p.partial) return rc;
    const int64_t parts = axis == AXIS_COL ? (m + p.rows - 1) / p.rows : (n + DACT_COLS - 1) / DACT_COLS;
    const int64_t len = axis == AXIS_COL ? n : m;
    return status(len % 8 == 0 ? launch_add_parts(dt, p.partial, parts, len, dbias, pdl, s)
                               : launch_sum_parts_f32(dt, p.partial, parts, len, dbias, pdl, s));      // ROW, odd m
}

}  // namespace

extern "C" {

int gemm_epi_rmsnorm(int64_t m, int64_t d, int dtype, int out_mode, float eps, const void *X, const void *R,
                     const void *gamma, void *S, void *Y, float *d_scale, float *d_amax, void *stream) {
    NormParams p{};
    int rc = norm_params(m, d, dtype, out_mode, eps, X, R, gamma, nullptr, S, Y, d_scale, d_amax, &p);
    if (rc != GEMM_EPI_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the amax word is this call's maximum: start it at 0 (the kernel max-reduces into it)
    const bool pdl = pdl_enabled();
    if (p.amax && (rc = status(launch_zero_word(p.amax, pdl, s))) != GEMM_EPI_OK) return rc;
    return status(launch_rmsnorm(dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16, out_mode, p, pdl, s));
}

int gemm_epi_layernorm(int64_t m, int64_t d, int dtype, int out_mode, float eps, const void *X, const void *R, const void *gamma,
                       const void *beta, void *S, void *Y, float *d_scale, float *d_amax, void *stream) {
    LnParams p{};
    int rc = norm_params(m, d, dtype, out_mode, eps, X, R, gamma, beta, S, Y, d_scale, d_amax, &p);
    if (rc != GEMM_EPI_OK) return rc;
    p.beta = beta;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pdl = pdl_enabled();
    if (p.amax && (rc = status(launch_zero_word(p.amax, pdl, s))) != GEMM_EPI_OK) return rc;
    return status(launch_layernorm(dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16, out_mode, p, pdl, s));
}

int gemm_epi_quant_rows(int64_t m, int64_t d, int dtype, int out_mode, const void *X, void *Q, float *d_scale, void *stream) {
    if (m <= 0 || d <= 0 || m > 0x7fffffffll || d > 0x7fffffffll) return GEMM_EPI_ERR_ARG;
    if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return GEMM_EPI_ERR_ARG;
    if (out_mode != GEMM_EPI_NORM_E4M3_ROWS && out_mode != GEMM_EPI_NORM_I8_ROWS) return GEMM_EPI_ERR_ARG;
    if (d % 16 != 0) return GEMM_EPI_ERR_ALIGN;
    if (!X || !Q || !d_scale) return GEMM_EPI_ERR_NULL;
    if (Q == X) return GEMM_EPI_ERR_ARG;                         // rows of another pitch
    if (!aligned(X, 16) || !aligned(Q, 16) || !aligned(d_scale, 4)) return GEMM_EPI_ERR_ALIGN;
    const int rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    NormParams p{};
    p.m = m;
    p.d = (int)d;
    p.x = X;
    p.y = Q;
    p.scale = d_scale;
    return status(launch_quant_rows(dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16, out_mode, p, pdl_enabled(),
                                    static_cast<cudaStream_t>(stream)));
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

int64_t gemm_epi_layernorm_workspace_bytes(int64_t m, int64_t d) {
    if (m <= 0 || d <= 0 || d > NORM_MAX_D || d % 8 != 0 || m > 0x7fffffffll) return 0;
    return ln_bwd_parts(m, d) * 2 * d * (int64_t)sizeof(float);
}

int gemm_epi_layernorm_bwd(int64_t m, int64_t d, int dtype, float eps, const void *dY, const void *S, const void *gamma,
                           const void *dS, void *dX, void *dgamma, void *dbeta, void *workspace, void *stream) {
    int rc = check_norm(m, d, dtype, eps, 8);
    if (rc != GEMM_EPI_OK) return rc;
    const int64_t parts = dgamma || dbeta ? ln_bwd_parts(m, d) : 0;
    if (!dY || !S || !gamma || !dX || (parts > 0 && !workspace)) return GEMM_EPI_ERR_NULL;
    if (dgamma && dgamma == dbeta) return GEMM_EPI_ERR_ARG;
    if (!aligned(dY, 16) || !aligned(S, 16) || !aligned(gamma, 16) || !aligned(dS, 16) || !aligned(dX, 16) ||
        !aligned(dgamma, 16) || !aligned(dbeta, 16) || !aligned(workspace, 16))
        return GEMM_EPI_ERR_ALIGN;
    rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int dt = dtype == GEMM_EPI_F16 ? DT_F16 : DT_BF16;
    LnBwdParams p{};
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
    p.dbeta = parts > 0 ? nullptr : dbeta;
    const bool pdl = pdl_enabled();
    rc = status(launch_layernorm_bwd(dt, p, pdl, s));
    if (rc != GEMM_EPI_OK || parts == 0) return rc;
    return status(launch_add_parts2(dt, p.partial, parts, 2 * d, dgamma, dbeta, d, pdl, s));
}

int64_t gemm_epi_ckpt_groups(int64_t n) { return n <= 0 || n > 0x7fffffffll ? 0 : ckpt_groups(n); }

int gemm_epi_ckpt_save(int64_t m, int64_t n, int dtype, int epilogue, const void *Z, void *H, int8_t *codes, uint8_t *exps,
                       void *stream) {
    int rc = check_ckpt(m, n, dtype, epilogue);
    if (rc != GEMM_EPI_OK) return rc;
    if (!Z || !codes || !exps) return GEMM_EPI_ERR_NULL;
    if (codes == Z || codes == H || exps == Z || exps == H || (const void *)exps == (const void *)codes) return GEMM_EPI_ERR_ARG;
    if (!aligned(Z, 16) || !aligned(H, 16) || !aligned(codes, 16)) return GEMM_EPI_ERR_ALIGN;
    rc = check_device();
    return rc != GEMM_EPI_OK ? rc : run_ckpt(true, m, n, dtype, epilogue, Z, H, codes, exps, stream);
}

int gemm_epi_ckpt_load(int64_t m, int64_t n, int dtype, int epilogue, const int8_t *codes, const uint8_t *exps, void *X,
                       void *stream) {
    int rc = check_ckpt(m, n, dtype, epilogue);
    if (rc != GEMM_EPI_OK) return rc;
    if (!X || !codes || !exps) return GEMM_EPI_ERR_NULL;
    if (codes == X || exps == X) return GEMM_EPI_ERR_ARG;
    if (!aligned(X, 16) || !aligned(codes, 16)) return GEMM_EPI_ERR_ALIGN;
    rc = check_device();
    return rc != GEMM_EPI_OK ? rc
                             : run_ckpt(false, m, n, dtype, epilogue, nullptr, X, const_cast<int8_t *>(codes),
                                        const_cast<uint8_t *>(exps), stream);
}

int64_t gemm_epi_dact_workspace_bytes(int64_t m, int64_t n, int bias_axis) {
    if (m <= 0 || n <= 0 || m > 0x7fffffffll || n > 0x7fffffffll) return 0;
    if (n % 8 != 0) return 0;
    if (bias_axis == GEMM_EPI_BIAS_ROW && dact_by_rows(m, n)) return 0;
    if (bias_axis == GEMM_EPI_BIAS_ROW) return (n + DACT_COLS - 1) / DACT_COLS * m * (int64_t)sizeof(float);
    if (bias_axis != GEMM_EPI_BIAS_COL) return 0;
    const int64_t rows = std::min(dact_rows(m, n, 3), dact_rows(m, n, 4));      // whatever the epilogue
    return rows >= m ? 0 : (m + rows - 1) / rows * n * (int64_t)sizeof(float);
}

int gemm_epi_dact(int64_t m, int64_t n, int dtype, int epilogue, int bias_axis, const void *dD, const void *Z,
                  const uint32_t *aux, void *dZ, void *dbias, void *workspace, void *stream) {
    if (m <= 0 || n <= 0 || m > 0x7fffffffll || n > 0x7fffffffll) return GEMM_EPI_ERR_ARG;
    if (dtype < GEMM_EPI_F16 || dtype > GEMM_EPI_E4M3) return GEMM_EPI_ERR_ARG;
    if (bias_axis != GEMM_EPI_BIAS_ROW && bias_axis != GEMM_EPI_BIAS_COL) return GEMM_EPI_ERR_ARG;
    const int act = dact_of_epilogue(epilogue);
    if (act < 0) return GEMM_EPI_ERR_ARG;
    if (n % 8 != 0) return GEMM_EPI_ERR_ALIGN;
    const bool mask = act == DACT_RELU_MASK;
    if (!dD || (mask && !aux) || (!mask && act != DACT_NONE && !Z)) return GEMM_EPI_ERR_NULL;
    if (act == DACT_NONE ? !dbias : !dZ) return GEMM_EPI_ERR_NULL;
    if (dbias && !workspace && dact_needs_workspace(m, n, dact_blocks(act, false), bias_axis)) return GEMM_EPI_ERR_NULL;
    if (act == DACT_NONE && dZ) return GEMM_EPI_ERR_ARG;          // dZ is dD itself
    if (!aligned(dD, 16) || (act != DACT_NONE && !mask && !aligned(Z, 16)) || (mask && !aligned(aux, 16)) ||
        !aligned(dZ, 16) || !aligned(dbias, 16) || !aligned(workspace, 16))
        return GEMM_EPI_ERR_ALIGN;
    const int rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    DactParams p{};
    p.dd = dD;
    p.z = Z;
    p.aux = reinterpret_cast<const uint8_t *>(aux);
    p.aux_pitch = gemm_epi_aux_pitch_bytes(n);
    p.dz = dZ;
    return run_dact(p, m, n, dtype, act, bias_axis, false, dbias, workspace, stream);
}

int gemm_epi_dact_ckpt(int64_t m, int64_t n, int dtype, int epilogue, int bias_axis, const void *dD, const int8_t *codes,
                       const uint8_t *exps, void *dZ, void *H, void *dbias, void *workspace, void *stream) {
    int rc = check_ckpt(m, n, dtype, epilogue);
    if (rc != GEMM_EPI_OK) return rc;
    if (bias_axis != GEMM_EPI_BIAS_ROW && bias_axis != GEMM_EPI_BIAS_COL) return GEMM_EPI_ERR_ARG;
    const int act = dact_of_epilogue(epilogue);
    if (act == DACT_NONE || act == DACT_RELU_MASK) return GEMM_EPI_ERR_ARG;      // nothing, or the mask, is kept of z
    if (!dD || !codes || !exps || !dZ) return GEMM_EPI_ERR_NULL;
    if (dbias && !workspace && dact_needs_workspace(m, n, dact_blocks(act, true), bias_axis)) return GEMM_EPI_ERR_NULL;
    if (H == dZ || codes == dZ || codes == H || exps == dZ || exps == H) return GEMM_EPI_ERR_ARG;
    if (!aligned(dD, 16) || !aligned(codes, 16) || !aligned(dZ, 16) || !aligned(H, 16) || !aligned(dbias, 16) || !aligned(workspace, 16))
        return GEMM_EPI_ERR_ALIGN;
    rc = check_device();
    if (rc != GEMM_EPI_OK) return rc;
    DactParams p{};
    p.dd = dD;
    p.codes = codes;
    p.exps = exps;
    p.dz = dZ;
    p.h = H;
    return run_dact(p, m, n, dtype, act, bias_axis, true, dbias, workspace, stream);
}

}  // extern "C"
