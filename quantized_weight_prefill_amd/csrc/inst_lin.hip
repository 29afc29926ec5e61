// inst_lin.hip -- one (format, dtype, activation layout, epilogue)
// instantiation of the linear layer's kernels: the rungs of inst_fp.hip with
// bias, activation, residual and gating applied to the accumulators; the
// build compiles this file once per combination with QG_FMT, QG_DT, QG_XL and
// QG_EPI defined.
#include "kernels_fp.h"

#if !defined(QG_FMT) || !defined(QG_DT) || !defined(QG_XL) || !defined(QG_EPI)
#error "inst_lin.hip is compiled with -DQG_FMT=<format> -DQG_DT=<dtype> -DQG_XL=<layout> -DQG_EPI=<epilogue>"
#endif

namespace qg {
template hipError_t launch_fd<QG_FMT, QG_DT, QG_XL, QG_EPI>(const Plan &, const Args &, hipStream_t);
}  // namespace qg
