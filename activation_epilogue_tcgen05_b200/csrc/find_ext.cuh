// find_ext.cuh -- lookup of the kernels with the extended epilogue (residual, scales by row);
// included only by the inst_*_ext.cu units that instantiate them.  The bias axis is a run-time
// choice in these kernels, and EPI_NONE runs EPI_BIAS without a bias.
#pragma once
#include "kernels.h"

namespace gemm_epi {

template <int DTV, bool Q>
struct TcFindExt {
    template <int CG, int EPI, bool BMN, int BN>
    static bool leaf(TcLauncher *l, KernelInfo *i) {
        constexpr int ES = dt_size(DTV);
        constexpr int STG = tc_stages(tc_katoms(128 * 128 + (BN / CG) * 128) * (128 * 128 + (BN / CG) * 128));
        if constexpr ((BMN && (BN / CG) % (128 / ES) != 0) || (BN == 512 && (CG != 2 || Q || DTV == DT_I8))) {
            return false;     // as for the plain kernels; no 512-wide tiles of 8-bit integers, whose mainloop is e4m3's
        } else {
            using C = TcCfg<DTV, EPI, AXIS_COL, BMN, BN, CG, STG, Q, false, true>;
            *l = &launch_tc<C>;
            *i = tc_info<C>();
            return true;
        }
    }
    template <int CG, int EPI, bool BMN>
    static bool width(int bn, TcLauncher *l, KernelInfo *i) {
        switch (bn) {
        case 128: return leaf<CG, EPI, BMN, 128>(l, i);
        case 256: return leaf<CG, EPI, BMN, 256>(l, i);
        case 512: return leaf<CG, EPI, BMN, 512>(l, i);
        }
        return false;
    }
    template <int EPI>
    static bool of(int cg, bool bmn, int bn, TcLauncher *l, KernelInfo *i) {
        if (cg == 1) return bmn ? width<1, EPI, true>(bn, l, i) : width<1, EPI, false>(bn, l, i);
        return bmn ? width<2, EPI, true>(bn, l, i) : width<2, EPI, false>(bn, l, i);
    }
    static bool find(int cg, int epi, bool bmn, int bn, TcLauncher *l, KernelInfo *i) {
        switch (epi) {
        case EPI_NONE: case EPI_BIAS: return of<EPI_BIAS>(cg, bmn, bn, l, i);
        case EPI_RELU: return of<EPI_RELU>(cg, bmn, bn, l, i);
        case EPI_GELU: return of<EPI_GELU>(cg, bmn, bn, l, i);
        }
        if constexpr (!Q) {
            if (epi == EPI_RELU_AUX) return of<EPI_RELU_AUX>(cg, bmn, bn, l, i);
            if (epi == EPI_TANH) return of<EPI_TANH>(cg, bmn, bn, l, i);
        }
        return false;
    }
};

template <int DTV, bool Q>
struct SkFindExt {
    template <int EPI, bool WMN, int NM>
    static bool leaf(SkLauncher *l, KernelInfo *i) {
        using C = SkCfg<DTV, EPI, AXIS_COL, WMN, NM, sk_stages(NM), Q, true>;
        *l = &launch_sk<C>;
        *i = sk_info<C>();
        return true;
    }
    template <int EPI, bool WMN>
    static bool rows(int nm, SkLauncher *l, KernelInfo *i) {
        switch (nm) {
        case 16: return leaf<EPI, WMN, 16>(l, i);
        case 32: return leaf<EPI, WMN, 32>(l, i);
        case 64: return leaf<EPI, WMN, 64>(l, i);
        case 128: return leaf<EPI, WMN, 128>(l, i);
        }
        return false;
    }
    template <int EPI>
    static bool of(bool wmn, int nm, SkLauncher *l, KernelInfo *i) {
        return wmn ? rows<EPI, true>(nm, l, i) : rows<EPI, false>(nm, l, i);
    }
    static bool find(int epi, bool wmn, int nm, SkLauncher *l, KernelInfo *i) {
        switch (epi) {
        case EPI_NONE: case EPI_BIAS: return of<EPI_BIAS>(wmn, nm, l, i);
        case EPI_RELU: return of<EPI_RELU>(wmn, nm, l, i);
        case EPI_GELU: return of<EPI_GELU>(wmn, nm, l, i);
        }
        if constexpr (!Q) {
            if (epi == EPI_RELU_AUX) return of<EPI_RELU_AUX>(wmn, nm, l, i);
            if (epi == EPI_TANH) return of<EPI_TANH>(wmn, nm, l, i);
        }
        return false;
    }
};

}  // namespace gemm_epi
