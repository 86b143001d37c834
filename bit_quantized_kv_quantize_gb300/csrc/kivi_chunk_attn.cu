// kivi_chunk_attn.cu -- plan and launch of the chunk attention
// (kivi_chunk_attn_impl.cuh).
#include <climits>
#include <cstdlib>
#include <cstring>

#include "kivi_chunk_attn_impl.cuh"

// (kivi_chunk_few.cu)
cudaError_t kivi_launch_chunk_few(const KiviGeom &, const KiviDev &, const __half *, const __half *, const __half *,
                                  __half *, ChunkArgs &, int, cudaStream_t);

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
    const int hg = a.hg;
    cudaError_t e = make_tile_map(&tk, K, rows, D, kCkKeys);
    if (e == cudaSuccess && kCkRows % hg == 0)
        e = make_group_rows_map(&tq, Q, (long long)g.b * g.h, hg, a.n_stride, D);
    if (e == cudaSuccess) e = make_tile_map(&tv, V, rows, D, kCkKeys);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    chunk_attn_kernel<D><<<ctas, kCkThreads, smem, st>>>(g, dv, Q, K, V, O, tq, tk, tv, a);
    return cudaGetLastError();
}

}  // namespace

size_t kivi_chunk_partial_floats(const KiviGeom &g, const ChunkPlan &plan, int num_sms) {
    return (size_t)2 * num_sms * (plan.few ? kFewRows : kCkTileRows) * (g.d + 2);
}

bool kivi_plan_units(int b, int h, ChunkArgs &a, int num_sms, int lead, int least, int *ctas, bool *join) {
    long long items = 0, U = 0;
    for (int i = 0; i < b; ++i) {
        const int mt = chunk_row_tiles(a, i);
        long long u = 0;
        for (int m = 0; m < mt; ++m) u += lead + chunk_tiles(a, i, m);
        U += u * h;
        items += (long long)mt * h;
    }
    // One CTA an SM, but no share below `least` units unless the row tiles
    // are that short: cutting them finer costs more than it shortens (the
    // join's launch too: row tiles of up to 3 lead units are not cut while
    // the SMs suffice for them).
    const long long sms = num_sms < kCkMaxCtas ? num_sms : kCkMaxCtas;
    const long long want = U > 3 * lead * items && U / least > items ? U / least : items;
    *ctas = (int)(want < sms ? want : sms);
    if (U / *ctas >= INT_MAX) return false;   // (CkWalk counts them)
    // each CTA's first unit, and whether one lies behind the first key tile of
    // a row tile (whose partials are then joined)
    *join = false;
    long long P = 0;   // the first unit of (i, m)
    int c = 0;
    for (int i = 0; i < b; ++i)
        for (int m = 0; m < chunk_row_tiles(a, i); ++m) {
            const int w = lead + chunk_tiles(a, i, m);
            const long long end = P + (long long)h * w;
            for (; c < *ctas && (long long)c * U / *ctas < end; ++c) {
                const long long u = (long long)c * U / *ctas;
                a.cta[c] = ChunkPos{u, i, m, (int)((u - P) / w), (int)((u - P) % w)};
                *join |= a.cta[c].o > lead;
            }
            P = end;
        }
    a.cta[*ctas] = ChunkPos{U, 0, 0, 0, 0};
    return true;
}

bool kivi_plan_chunk_attn(const KiviGeom &g, ChunkArgs &a, int num_sms, ChunkPlan *plan) {
    const int hg = a.hq / g.h;
    a.hg = hg;
    a.hg_mul = (unsigned)(((1ull << 32) + hg - 1) / hg);
    int maxrows = 0, end = 0, seen = 0;   // seen: the most blocks that a sequence sees
    for (int i = 0; i < g.b; ++i) {
        maxrows = a.n[i] * hg > maxrows ? a.n[i] * hg : maxrows;
        end = a.T[i] + a.n[i] > end ? a.T[i] + a.n[i] : end;
    }
    *plan = ChunkPlan{false, false, 0};
    if (maxrows == 0) return true;
    // a window that no position reaches is none (and would pass 32 bits below
    // the first positions)
    if (a.vis.window >= end) a.vis = Visible{0, 0};
    for (int i = 0; i < g.b; ++i)
        if (a.n[i] > 0) {
            const int x = visible_blocks(a.vis, a.T[i]).virt((a.T[i] + a.n[i] - 1) / KIVI_KBLK + 1);
            seen = x > seen ? x : seen;
        }
    // Up to 16 rows a kv head over 32 blocks or more: the transposed kernel,
    // whose work follows the rows.  It and 256-row tiles, 16 rows over a cache
    // of 8 sequences of 8 heads, in microseconds: 32k tokens 151 and 208, 8000
    // 53 and 62, 2000 30 and 33, 1000 27 and 26, 100 15 and 10.  (32 rows, in a
    // variant for them: 32k 192 and 209, 4000 49 and 42.)
    const bool few = maxrows <= kFewRows && seen >= 32;
    a.tile_rows = few ? kFewRows : kCkTileRows;
    a.tile_blocks = few ? 2 : 1;
    int ctas = 0;
    bool join = false;
    if (!kivi_plan_units(g.b, g.h, a, num_sms, kCkLead, 2 * kCkLead, &ctas, &join)) return false;
    const char *quit = getenv("KIVI_CHUNK_QUIT");
    a.quit = quit ? atoi(quit) : INT_MAX;
    *plan = ChunkPlan{few, join, ctas};
    return true;
}

cudaError_t kivi_launch_chunk_attn(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                   const __half *V, __half *O, ChunkArgs &a, const ChunkPlan &plan, float *partials,
                                   int num_sms, cudaStream_t st) {
    if (plan.ctas == 0) return cudaSuccess;
    if (g.d != 64 && g.d != 128) return cudaErrorInvalidValue;
    if ((long long)g.b * g.h * a.n_stride >= (1LL << 31)) return cudaErrorInvalidValue;   // TMA row coordinates
    a.acc = partials;
    a.ml = partials + (size_t)2 * num_sms * a.tile_rows * g.d;
    cudaError_t e = plan.few ? kivi_launch_chunk_few(g, dv, Q, K, V, O, a, plan.ctas, st)
                    : g.d == 64 ? launch_chunk<64>(g, dv, Q, K, V, O, a, plan.ctas, st)
                                : launch_chunk<128>(g, dv, Q, K, V, O, a, plan.ctas, st);
    if (e != cudaSuccess || !plan.join) return e;
    const unsigned blocks = (unsigned)(plan.ctas - 1) * (a.tile_rows / kJoinRows);
    if (g.d == 64) chunk_join_kernel<64><<<blocks, 256, 0, st>>>(O, a);
    else chunk_join_kernel<128><<<blocks, 256, 0, st>>>(O, a);
    return cudaGetLastError();
}
