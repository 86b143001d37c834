// kivi_prefill_attn.cu -- launch of the causal prefill attention with its
// pack epilogue (kivi_prefill_attn_impl.cuh).
#include "kivi_prefill_attn_impl.cuh"

cudaError_t kivi_launch_prefill_attn_win(const KiviGeom &, const KiviDev &, const __half *, const __half *,
                                         const __half *, __half *, const SeqLens &, int, int, int, const Visible &,
                                         cudaStream_t);

cudaError_t kivi_launch_prefill_attn(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                     const __half *V, __half *O, const SeqLens &lens, int t_stride, int hq,
                                     cudaStream_t st, Visible vis) {
    if (g.G > 64 || (g.d != 64 && g.d != 128)) return cudaErrorInvalidValue;
    int maxt = 0;
    for (int i = 0; i < g.b; ++i) maxt = lens.t[i] > maxt ? lens.t[i] : maxt;
    if (maxt > 0 && ((long long)g.b * hq * t_stride >= (1LL << 31))) return cudaErrorInvalidValue;   // TMA row coordinates
    return vis.window > 0 ? kivi_launch_prefill_attn_win(g, dv, Q, K, V, O, lens, t_stride, hq, maxt, vis, st)
                          : launch_shape<false>(g, dv, Q, K, V, O, lens, t_stride, hq, maxt, vis, st);
}
