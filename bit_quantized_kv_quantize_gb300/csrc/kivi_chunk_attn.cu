// kivi_chunk_attn.cu -- plan and launch of the chunk attention
// (kivi_chunk_attn_impl.cuh).
#include <cstring>

#include "kivi_chunk_attn_impl.cuh"

namespace {

template <int D>
cudaError_t launch_chunk(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K, const __half *V,
                         __half *O, ChunkArgs &a, int ctas, cudaStream_t st) {
    const size_t fixed = (size_t)2 * kCkRows * D * 2 + (size_t)2 * kCkStages * kCkKeys * D * 2 + kCkOut;
    a.rs = (int)((226 * 1024 - fixed) / g.rec_bytes);
    if (a.rs > kCkMaxRaw) a.rs = kCkMaxRaw;
    if (a.rs < 2) return cudaErrorInvalidValue;
    const size_t smem = fixed + (size_t)a.rs * g.rec_bytes;
    CUtensorMap tq, tk, tv;
    memset(&tq, 0, sizeof tq);   // unused with a head group that does not divide 128
    const long long rows = (long long)g.b * g.h * a.n_stride;
    const int hg = a.hq / g.h;
    cudaError_t e = make_tile_map(&tk, K, rows, D, kCkKeys);
    if (e == cudaSuccess && kCkRows % hg == 0)
        e = make_group_rows_map(&tq, Q, (long long)g.b * g.h, hg, a.n_stride, D);
    if (e == cudaSuccess) e = make_tile_map(&tv, V, rows, D, kCkKeys);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    chunk_attn_kernel<D><<<ctas, kCkThreads, smem, st>>>(g, dv, Q, K, V, O, tq, tk, tv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // does a CTA's range start behind the first tile of a row tile?
    const long long U = a.ustart[g.b];
    bool join = false;
    long long P = 0;   // the first unit of (i, m)
    for (int i = 0, c = 1; i < g.b && !join; ++i)
        for (int m = 0; m < chunk_row_tiles(a.n[i], hg) && !join; ++m) {
            const int w = kCkLead + chunk_tiles(a, i, m, hg);
            const long long end = P + (long long)g.h * w;
            for (; c < ctas && (long long)c * U / ctas < end; ++c) join |= ((long long)c * U / ctas - P) % w > kCkLead;
            P = end;
        }
    if (!join) return cudaSuccess;
    chunk_join_kernel<D><<<(ctas - 1) * (kCkTileRows / 32), 256, 0, st>>>(g, O, a, ctas);
    return cudaGetLastError();
}

}  // namespace

size_t kivi_chunk_partial_floats(int d, int num_sms) {
    return d > 128 ? 0 : (size_t)2 * num_sms * kCkTileRows * (d + 2);
}

cudaError_t kivi_launch_chunk_attn(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                   const __half *V, __half *O, ChunkArgs &a, float *partials, int num_sms,
                                   cudaStream_t st) {
    if (g.d != 64 && g.d != 128) return cudaErrorInvalidValue;
    if ((long long)g.b * g.h * a.n_stride >= (1LL << 31)) return cudaErrorInvalidValue;   // TMA row coordinates
    const int hg = a.hq / g.h;
    int maxrows = 0;
    long long items = 0;
    a.ustart[0] = 0;
    for (int i = 0; i < g.b; ++i) {
        const int mt = chunk_row_tiles(a.n[i], hg);
        long long u = 0;
        for (int m = 0; m < mt; ++m) u += kCkLead + chunk_tiles(a, i, m, hg);
        a.ustart[i + 1] = a.ustart[i] + u * g.h;
        items += (long long)mt * g.h;
        maxrows = a.n[i] * hg > maxrows ? a.n[i] * hg : maxrows;
    }
    if (maxrows == 0) return cudaSuccess;
    // One CTA an SM; where the row tiles are short (a CTA's share below 16
    // units), one a row tile, or one a few of them: cutting them would cost
    // more than it balances.
    const long long U = a.ustart[g.b];
    long long ctas = num_sms;
    if (U < 16 * ctas) ctas = items < ctas ? items : ctas;
    a.acc = partials;
    a.ml = partials + (size_t)2 * num_sms * kCkTileRows * g.d;
    return g.d == 64 ? launch_chunk<64>(g, dv, Q, K, V, O, a, (int)ctas, st)
                     : launch_chunk<128>(g, dv, Q, K, V, O, a, (int)ctas, st);
}
