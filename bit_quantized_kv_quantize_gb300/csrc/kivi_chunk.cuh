// kivi_chunk.cuh -- what the host and the kernels of the chunk calls share:
// a chunk's arguments, its counters afterwards, and the launchers.
#pragma once
#include "kivi_internal.cuh"

// One chunk call (kernel parameters): per sequence the cache's counters and
// the chunk's tokens, from the host mirror; the attention's work list: the
// units are each row tile of each kv head (kCkLead, then one a key tile; by
// sequence, row tile, head), and CTA c takes those from cta[c] up to
// cta[c + 1].
constexpr int kCkMaxCtas = 256;
struct ChunkPos {
    long long u;    // units before it
    int i, m, j;    // the row tile it lies in: sequence, row tile, kv head
    int o;          // its offset there
};
struct ChunkArgs {
    int hq, hg, n_stride;         // hg: query heads a kv head
    unsigned hg_mul;              // ceil(2^32 / hg): x / hg = umulhi(x, hg_mul) for x < 2^29 (hg <= 8)
    int rs;           // record stages
    int tile_rows, tile_blocks;   // rows of a row tile, 64-token blocks of a key tile
    Visible vis;
    int quit;         // (tests) a warp gives up: with few rows the copying one after so many records, else
                      // the dequantizing ones but the first at once; INT_MAX: none does
    float *acc, *ml;  // partials: [2 CTAs][tile_rows][d] and [2 CTAs][tile_rows][2]
    ChunkPos cta[kCkMaxCtas + 1];
    int T[KIVI_MAX_BATCH], Tqk[KIVI_MAX_BATCH], Tqv[KIVI_MAX_BATCH], n[KIVI_MAX_BATCH];
};

constexpr int kFewRows = 16;  // rows of the row tiles for few rows
constexpr int kCkLead = 4;   // units that stand for a row tile's fixed cost

// x / hg
__host__ __device__ __forceinline__ int chunk_div(const ChunkArgs &a, int x) {
#ifdef __CUDA_ARCH__
    return a.hg == 1 ? x : (int)__umulhi((unsigned)x, a.hg_mul);
#else
    return x / a.hg;
#endif
}
// Row tiles of sequence i's kv heads, and the 64-token blocks and key tiles
// that its row tile m sees.
__host__ __device__ __forceinline__ int chunk_row_tiles(const ChunkArgs &a, int i) {
    return (a.n[i] * a.hg + a.tile_rows - 1) / a.tile_rows;
}
__host__ __device__ __forceinline__ int chunk_blocks(const ChunkArgs &a, int i, int m) {
    const int r0 = chunk_div(a, m * a.tile_rows), r1 = chunk_div(a, m * a.tile_rows + a.tile_rows - 1);
    const int last = r1 < a.n[i] - 1 ? r1 : a.n[i] - 1;
    return visible_blocks(a.vis, a.T[i] + r0).virt((a.T[i] + last) / KIVI_KBLK + 1);
}
__host__ __device__ __forceinline__ int chunk_tiles(const ChunkArgs &a, int i, int m) {
    return (chunk_blocks(a, i, m) + a.tile_blocks - 1) / a.tile_blocks;   // 1 or 2 blocks a tile
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

// How a chunk's attention runs.
struct ChunkPlan {
    bool few;   // the kernel for few rows
    bool join;  // row tiles are cut: partials, and the kernel that joins them
    int ctas;   // 0: nothing to do
};
// floats of the partials that a plan's row tiles leave (two a CTA)
size_t kivi_chunk_partial_floats(const KiviGeom &g, const ChunkPlan &plan, int num_sms);
// Plans the attention of the chunk (kivi_chunk_attn.cu).  a: hq, n_stride,
// vis, T, Tqk, Tqv and n; the work list is added.  False if a CTA's share
// would pass 32 bits.
bool kivi_plan_chunk_attn(const KiviGeom &g, ChunkArgs &a, int num_sms, ChunkPlan *plan);
// ... and launches it.  partials: not used without a join.  d in {64, 128}
// (cudaErrorInvalidValue otherwise).
cudaError_t kivi_launch_chunk_attn(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K,
                                   const __half *V, __half *O, ChunkArgs &a, const ChunkPlan &plan, float *partials,
                                   int num_sms, cudaStream_t st);
// The append of the chunk (kivi_chunk_append.cu); the counters after it go to
// nxt ([3][b], the other counter set).
cudaError_t kivi_launch_append_chunk(const KiviGeom &g, const KiviDev &dv, const __half *K, const __half *V,
                                     const ChunkArgs &a, int *nxt, cudaStream_t st);
