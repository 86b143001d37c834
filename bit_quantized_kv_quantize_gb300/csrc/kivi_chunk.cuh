// kivi_chunk.cuh -- what the host and the kernels of the chunk calls share:
// a chunk's arguments, its counters afterwards, and the launchers.
#pragma once
#include "kivi_internal.cuh"

// One chunk call (kernel parameters): per sequence the cache's counters and
// the chunk's tokens, from the host mirror; the attention's work list:
// sequence i's CTAs are [start[i], start[i + 1]), ordered (kv head, row tile,
// piece of the tile's tokens).
struct ChunkArgs {
    int hq, n_stride;
    int rs;           // record stages
    Visible vis;
    float *acc, *ml;  // split partials: [CTA][rows][d] and [CTA][rows][2]
    int T[KIVI_MAX_BATCH], Tqk[KIVI_MAX_BATCH], Tqv[KIVI_MAX_BATCH], n[KIVI_MAX_BATCH];
    int start[KIVI_MAX_BATCH + 1];
};

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
// ml, start.  d in {64, 128} (cudaErrorInvalidValue otherwise).
cudaError_t kivi_launch_chunk_attn(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                   const __half *V, __half *O, ChunkArgs &a, float *partials, int num_sms,
                                   cudaStream_t st);
// The append of the chunk (kivi_chunk_append.cu); the counters after it go to
// nxt ([3][b], the other counter set).
cudaError_t kivi_launch_append_chunk(const KiviGeom &g, const KiviDev &dv, const __half *K, const __half *V,
                                     const ChunkArgs &a, int *nxt, cudaStream_t st);
