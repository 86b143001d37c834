// kivi_decode_win_d128.cu -- decode-attention kernels for head dimension 128
// with a sliding window and sink tokens.
#include "kivi_decode_impl.cuh"

cudaError_t kivi_launch_decode_win_d128(const KiviGeom &g, const KiviDev &dv, const __half *q, int hq, __half *out,
                                       const DecodePlan &plan, const DecodeUnits &units, const Visible &vis,
                                       cudaStream_t st) {
    return launch_d<128, false, false, true>(g, dv, q, hq, out, plan, units, ProbsOut{nullptr, nullptr, 0}, st,
                                            FusedStep{nullptr, nullptr, nullptr}, vis);
}
