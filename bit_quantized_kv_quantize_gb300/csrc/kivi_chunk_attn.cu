// kivi_chunk_attn.cu -- plan and launch of the chunk attention
// (kivi_chunk_attn_impl.cuh).
#include "kivi_chunk_attn_impl.cuh"

namespace {

// Partials: two CTAs' worth of 128 rows an SM (or one of 256).
constexpr int kPartRowsPerSm = 256;

// Fixed cost of a piece (set-up, its first tile's latency, its result) and
// of the joining launch, in key tiles of one row tile.
constexpr int kPieceCost = 6, kJoinCost = 8;

}  // namespace

size_t kivi_chunk_partial_floats(int d, int num_sms) {
    return d > 128 ? 0 : (size_t)num_sms * kPartRowsPerSm * (d + 2);
}

cudaError_t kivi_launch_chunk_attn(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                   const __half *V, __half *O, ChunkArgs &a, float *partials, int num_sms,
                                   cudaStream_t st) {
    if (g.d != 64 && g.d != 128) return cudaErrorInvalidValue;
    const int hg = a.hq / g.h;
    int maxrows = 0;
    for (int i = 0; i < g.b; ++i) maxrows = a.n[i] * hg > maxrows ? a.n[i] * hg : maxrows;
    if (maxrows == 0) return cudaSuccess;
    // two 128-row slots a CTA share each restored tile; one when the rows fit
    const int NH = maxrows > kCkRows ? 2 : 1, CR = NH * kCkRows;
    int nt[KIVI_MAX_BATCH];   // the most key tiles of a row tile of sequence i
    long long items = 0;
    int maxnt = 1;
    for (int i = 0; i < g.b; ++i) {
        nt[i] = 1;
        const int rows = a.n[i] * hg;
        for (int r0 = 0; r0 < rows; r0 += CR) {
            const int p1 = a.T[i] + ((r0 + CR < rows ? r0 + CR : rows) - 1) / hg;
            const int c = visible_blocks(a.vis, a.T[i] + r0 / hg).virt(p1 / kCkKeys + 1);
            nt[i] = c > nt[i] ? c : nt[i];
        }
        items += (long long)g.h * ((rows + CR - 1) / CR);
        maxnt = nt[i] > maxnt ? nt[i] : maxnt;
    }
    // Tiles a piece: no split unless it shortens the slowest SM's work (waves
    // of CTAs, one an SM, times a piece's tiles and fixed cost)
    auto pieces = [&](int P) {
        long long c = 0;
        for (int i = 0; i < g.b; ++i)
            c += (long long)g.h * ((a.n[i] * hg + CR - 1) / CR) * ((nt[i] + P - 1) / P);
        return c;
    };
    int best = maxnt;
    long long cost = (items + num_sms - 1) / num_sms * (long long)(maxnt + kPieceCost);
    const long long cap = (long long)num_sms * kPartRowsPerSm / CR;
    for (int waves = 1; waves <= 2; ++waves) {
        const long long limit = (long long)num_sms * waves < cap ? (long long)num_sms * waves : cap;
        if (pieces(maxnt) > limit) continue;
        int lo = 1, hi = maxnt;   // the smallest P within the limit
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (pieces(mid) <= limit) hi = mid; else lo = mid + 1;
        }
        if (lo >= maxnt) continue;
        const long long c = (long long)waves * (lo + kPieceCost) + kJoinCost;
        if (c < cost) {
            cost = c;
            best = lo;
        }
    }
    a.start[0] = 0;
    long long total = 0;
    for (int i = 0; i < g.b; ++i) {
        total += (long long)g.h * ((a.n[i] * hg + CR - 1) / CR) * ((nt[i] + best - 1) / best);
        if (total >= (1LL << 31)) return cudaErrorInvalidValue;
        a.start[i + 1] = (int)total;
    }
    a.acc = partials;
    a.ml = partials + (size_t)num_sms * kPartRowsPerSm * g.d;
    const bool join = best < maxnt;
    const int ctas = (int)total;
    if (g.d == 64)
        return NH == 1 ? launch_chunk<64, 1>(g, dv, Q, K, V, O, a, ctas, maxrows, join, st)
                       : launch_chunk<64, 2>(g, dv, Q, K, V, O, a, ctas, maxrows, join, st);
    return NH == 1 ? launch_chunk<128, 1>(g, dv, Q, K, V, O, a, ctas, maxrows, join, st)
                   : launch_chunk<128, 2>(g, dv, Q, K, V, O, a, ctas, maxrows, join, st);
}
