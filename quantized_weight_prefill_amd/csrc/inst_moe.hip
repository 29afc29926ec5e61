// inst_moe.hip -- the few-token mixture-of-experts kernels of one weight
// format; the build compiles this file once per format with QG_FMT defined.
#include "kernels_moe.h"

#if !defined(QG_FMT)
#error "inst_moe.hip is compiled with -DQG_FMT=<format>"
#endif

namespace qg {

template <int FMT>
hipError_t launch_moe_up(int dtype, dim3 grid, const MoeArgs &m, hipStream_t s)
{
    const dim3 block(64 * kMoeUpWaves);
    if (dtype == DT_F16 && !m.blocked) hipLaunchKernelGGL((k_moe_up<FMT, DT_F16, false>), grid, block, 0, s, m);
    else if (dtype == DT_F16) hipLaunchKernelGGL((k_moe_up<FMT, DT_F16, true>), grid, block, 0, s, m);
    else if (!m.blocked) hipLaunchKernelGGL((k_moe_up<FMT, DT_BF16, false>), grid, block, 0, s, m);
    else hipLaunchKernelGGL((k_moe_up<FMT, DT_BF16, true>), grid, block, 0, s, m);
    return hipGetLastError();
}

template <int FMT, int PN, bool BLOCKED>
void launch_down(int dtype, dim3 grid, const MoeArgs &m, hipStream_t s)
{
    const dim3 block(64 * kMoeDownWaves);
    const size_t lds = moe_down_lds(m.g.M, m.g.E, m.parts, PN, moe_down_rows(BLOCKED));
    if (dtype == DT_F16) hipLaunchKernelGGL((k_moe_down<FMT, DT_F16, PN, BLOCKED>), grid, block, lds, s, m);
    else hipLaunchKernelGGL((k_moe_down<FMT, DT_BF16, PN, BLOCKED>), grid, block, lds, s, m);
}

template <int FMT>
hipError_t launch_moe_down(int dtype, int pn, dim3 grid, const MoeArgs &m, hipStream_t s)
{
    if (pn == 1 && !m.blocked) launch_down<FMT, 1, false>(dtype, grid, m, s);
    else if (pn == 1) launch_down<FMT, 1, true>(dtype, grid, m, s);
    else if (!m.blocked) launch_down<FMT, 2, false>(dtype, grid, m, s);
    else launch_down<FMT, 2, true>(dtype, grid, m, s);
    return hipGetLastError();
}

template hipError_t launch_moe_up<QG_FMT>(int, dim3, const MoeArgs &, hipStream_t);
template hipError_t launch_moe_down<QG_FMT>(int, int, dim3, const MoeArgs &, hipStream_t);

}  // namespace qg
