// kivi_chunk.cuh -- what the host and the kernels of the chunk calls share:
// a chunk's arguments, its counters afterwards, and the launchers.
#pragma once
#include "kivi_internal.cuh"

// One chunk call (kernel parameters): per sequence the cache's counters and
// the chunk's tokens, from the host mirror; the attention's work list: the
// units of sequence i (each row tile of each kv head: kCkLead, then one a key
// tile; ordered by row tile, then head) are [ustart[i], ustart[i + 1]).
struct ChunkArgs {
    int hq, n_stride;
    int rs;           // record stages
    Visible vis;
    float *acc, *ml;  // partials: [2 CTAs][kCkTileRows][d] and [2 CTAs][kCkTileRows][2]
    int T[KIVI_MAX_BATCH], Tqk[KIVI_MAX_BATCH], Tqv[KIVI_MAX_BATCH], n[KIVI_MAX_BATCH];
    long long ustart[KIVI_MAX_BATCH + 1];
};

constexpr int kCkTileRows = 256;   // rows of a row tile
constexpr int kCkLead = 4;         // units that stand for a row tile's fixed cost

// Row tiles of a kv head with hg query heads, and the key tiles (64-token
// blocks) that row tile m of sequence i sees.
__host__ __device__ __forceinline__ int chunk_row_tiles(int n, int hg) {
    return (n * hg + kCkTileRows - 1) / kCkTileRows;
}
__host__ __device__ __forceinline__ int chunk_tiles(const ChunkArgs &a, int i, int m, int hg) {
    const int r0 = m * kCkTileRows / hg, r1 = (m * kCkTileRows + kCkTileRows - 1) / hg;
    const int last = r1 < a.n[i] - 1 ? r1 : a.n[i] - 1;
    return visible_blocks(a.vis, a.T[i] + r0).virt((a.T[i] + last) / KIVI_KBLK + 1);
}
// Counters after n one-token appends (item 4's lazy maintenance: a full key
// window flushes, and a value queue of R + 1 pops, at the start of the next
// append).
__host__ __device__ __forceinline__ int chunk_tqk(int T, int Tqk, int n, int R) {
    const int f = (T + n - 1) / R * R;
    return n > 0 && f > Tqk ? f : Tqk;
}
__host__ __device__ __forceinline__ int chunk_tqv(int T, int Tqv, int n, int R) {
    const int f = T + n - R - 1;
    return n > 0 && f > Tqv ? f : Tqv;
}

// floats of the attention's partials buffer of a cache with head dimension d
size_t kivi_chunk_partial_floats(int d, int num_sms);
// The attention of the chunk (kivi_chunk_attn.cu).  a: everything but rs, acc,
// ml, ustart.  d in {64, 128} (cudaErrorInvalidValue otherwise).
cudaError_t kivi_launch_chunk_attn(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                   const __half *V, __half *O, ChunkArgs &a, float *partials, int num_sms,
                                   cudaStream_t st);
// The append of the chunk (kivi_chunk_append.cu); the counters after it go to
// nxt ([3][b], the other counter set).
cudaError_t kivi_launch_append_chunk(const KiviGeom &g, const KiviDev &dv, const __half *K, const __half *V,
                                     const ChunkArgs &a, int *nxt, cudaStream_t st);
