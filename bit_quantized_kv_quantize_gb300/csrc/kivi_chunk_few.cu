// kivi_chunk_few.cu -- launch of the chunk attention for few query rows
// (kivi_chunk_few_impl.cuh).
#include "kivi_chunk_few_impl.cuh"

namespace {

template <int D>
cudaError_t launch_few(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K, const __half *V,
                       __half *O, ChunkArgs &a, int ctas, cudaStream_t st) {
    const size_t fixed = (size_t)kFwStages * (fw_kb(D) + fw_vb(D)) + (size_t)kFwRows * D * 2 + (size_t)kFwBufs * kFwKeys * kFwRows * 2;
    a.rs = (int)((224 * 1024 - fixed) / g.rec_bytes);
    if (a.rs > kFwMaxRaw) a.rs = kFwMaxRaw;
    if (a.rs < 4) return cudaErrorInvalidValue;
    const size_t smem = fixed + (size_t)a.rs * g.rec_bytes;
    cudaError_t e = cudaFuncSetAttribute(chunk_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    chunk_few_kernel<D><<<ctas, kFwThreads, smem, st>>>(g, dv, Q, K, V, O, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t kivi_launch_chunk_few(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                  const __half *V, __half *O, ChunkArgs &a, int ctas, cudaStream_t st) {
    return g.d == 64 ? launch_few<64>(g, dv, Q, K, V, O, a, ctas, st) : launch_few<128>(g, dv, Q, K, V, O, a, ctas, st);
}
