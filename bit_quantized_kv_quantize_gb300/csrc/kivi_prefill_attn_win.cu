// kivi_prefill_attn_win.cu -- the causal prefill attention with a sliding
// window and sink tokens (kivi_prefill_attn_impl.cuh).
#include "kivi_prefill_attn_impl.cuh"

cudaError_t kivi_launch_prefill_attn_win(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                         const __half *V, __half *O, const SeqLens &lens, int t_stride, int hq,
                                         int maxt, const Visible &vis, cudaStream_t st) {
    return launch_shape<true>(g, dv, Q, K, V, O, lens, t_stride, hq, maxt, vis, st);
}
