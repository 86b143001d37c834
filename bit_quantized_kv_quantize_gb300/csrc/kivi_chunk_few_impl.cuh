// kivi_chunk_few_impl.cuh -- chunk attention where each kv head has few query
// rows (a speculative step's tokens, a short last piece): the transposed form
// of the chunk attention (kivi_chunk_attn_impl.cuh has the mathematics).
//
// With 128 query rows on the MMA's M side, a few rows leave most of the tensor
// cores' and the softmax's work padding, and four warps that restore each
// tile between them set its time however few the rows (215 us where this
// kernel takes 148).  Here the tokens are on the M side and up to 16 rows
// on N:
//   S^T [128 tokens x N] = K^ Q^T,   O^T [d x N] += V^^T P^T,
// so a tile of 128 tokens costs 16 MMAs of N columns, thread t of the softmax
// owns token t and computes N weights, and what remains is restoring the
// tile: the kernel is bound by the dequantizing warps' instructions (4.5 a
// pair of values; the SMs issue in 47 % of their cycles, HBM is at 19 %).
// Measured over 32k 2-bit tokens of 8 sequences of 8 heads (204 MB, 30 us at
// the copy rate), joining included: 148 us; over 2000 tokens 30 us.  (N = 32,
// for 32 rows: 190 us over 32k, 226 where 256-row tiles take 206 over 8k tokens
// of 32 sequences.)
//
// The softmax needs a row's maximum over the tile's tokens, which are spread
// over the threads.  It is not formed a tile: the weights are taken against
// the row's reference, and only when some score lies more than 2^8 above it
// (one vote of the four warps a tile) are the maxima formed (redux.f32 over
// the lanes, then the warps), the references raised, and O^T and the sums
// rescaled.  A thread keeps its own part of each row's sum; they are added up
// at the end of the segment.
//
// The order of the channels in K^ and Q, and of the tokens in V^ and P^T, is
// free as long as both operands keep it.  It is chosen so that a lane's
// unpacked values of a record are 16 consecutive bytes of a tile (8 channels
// of a token: fw_chan; 8 tokens of a channel: fw_tok), stored at once, where
// the natural order takes four stores.
//
// V^ is always the [channels][tokens] tile here (the MMA's A operand); fp16
// tokens of the windows and the chunk are written transposed, value by value
// (a few tiles of a sequence).  P^T goes through shared memory as the B
// operand (rows contiguous: a thread stores its token's N weights 16 bytes at
// a time, lane by lane, without bank conflicts).
#pragma once
#include "kivi_chunk_tiles.cuh"
#include "kivi_tcgen05.cuh"

namespace {

constexpr int kFwRows = kFewRows;
constexpr int kFwKeys = 128;    // tokens of a tile (two blocks)
constexpr int kFwStages = 2;    // K^ tiles, and V^ tiles, in flight
constexpr int kFwMaxRaw = 12;   // records in flight
// Dequantizing warps: four for K^ and four for V^, block b of a CTA to warp b
// mod 4 (a V^ stage is held until the softmax and O^T are through with it: K^
// must not wait for that).  A warp restores a whole block in a short loop: with
// a role a warp, straight-line code runs at the rate of instruction fetches
// (measured: 7 cycles an instruction when four warps shared a block, each
// running its part once).
constexpr int kFwDq = 4;
constexpr int kFwThreads = 32 * (4 + 2 * kFwDq + 3);
// S^T and P^T buffers: tiles that the softmax may be apart from either MMA
// (four hide the waits between the roles)
constexpr int kFwBufs = 4;
// Bytes from a 16-byte chunk to the next along a row of K^, and of V^^T: 32
// more than their rows take, so that the lanes of a store (2 rows of 4 chunks)
// fall in different banks; bytes of a tile.
constexpr int kFwKS = kFwKeys * 16 + 32;
__host__ __device__ constexpr int fw_vs(int D) { return D * 16 + 32; }
__host__ __device__ constexpr int fw_kb(int D) { return D / 8 * kFwKS; }
__host__ __device__ constexpr int fw_vb(int D) { return kFwKeys / 8 * fw_vs(D); }
constexpr float kFwUnset = 1e30f;   // s_ref of a row that has seen nothing

__device__ __forceinline__ float redux_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
// OR over the four softmax warps (which all come here every tile)
__device__ __forceinline__ bool fw_any(bool v) {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void fw_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

// Position of channel c in a row of K^ and Q, of token r in a row of V^^T and
// in P^T.
__device__ __forceinline__ int fw_chan(int c) {
    return (c & ~31) | ((c >> 1) & 3) << 3 | ((c >> 4) & 1) << 2 | ((c >> 3) & 1) << 1 | (c & 1);
}
__device__ __forceinline__ int fw_tok(int r) {
    return (r & ~31) | ((r >> 1) & 3) << 3 | ((r >> 4) & 1) << 2 | ((r >> 3) & 1) << 1 | (r & 1);
}

// K^ of a record's 64 tokens (rows of the tile from `tile` on), channels in
// fw_chan's order, by one warp: a turn restores 32 channels of 32 tokens, lane
// (gq, tq) the 8 channels at position 8 tq of tokens 8 pos + gq.  LG: log2 of
// the group size.
template <int D, int KB, int LG>
__device__ __forceinline__ void few_keys(unsigned char *tile, const unsigned char *rec) {
    constexpr int KC = 2 * D * KB * 4;          // code bytes
    constexpr int GH = LG >= 5 ? 1 : 2;         // groups 32 tokens span
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const unsigned char *pw = rec + lane * 16;
    const __half *ksz = reinterpret_cast<const __half *>(rec + KC) + tq * (D / 4);
    unsigned char *dst = tile + (size_t)tq * kFwKS + gq * 16;
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
        const int jp = k >> 1, th = k & 1;      // 32 channels, half of the tokens
        // words of 16-channel steps 2 jp, 2 jp + 1: [step][hh], the half's codes lowest
        uint32_t W[4];
        if (KB == 2) {
            const uint4 v = *reinterpret_cast<const uint4 *>(pw + jp * 512);
            W[0] = v.x >> (8 * th);
            W[1] = v.y >> (8 * th);
            W[2] = v.z >> (8 * th);
            W[3] = v.w >> (8 * th);
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(pw + jp * 1024);
            const uint4 u = *reinterpret_cast<const uint4 *>(pw + jp * 1024 + 512);
            W[0] = th ? v.y : v.x;
            W[1] = th ? v.w : v.z;
            W[2] = th ? u.y : u.x;
            W[3] = th ? u.w : u.z;
        }
        uint4 sv[GH], zv[GH];                   // the lane's 8 channels' scales and zeros
#pragma unroll
        for (int q = 0; q < GH; ++q) {
            const int row = LG >= 6 ? 0 : th * GH + q;
            sv[q] = *reinterpret_cast<const uint4 *>(ksz + 8 * jp + 2 * row * D);
            zv[q] = *reinterpret_cast<const uint4 *>(ksz + 8 * jp + (2 * row + 1) * D);
        }
        unsigned char *p = dst + jp * (4 * kFwKS) + th * 512;
#pragma unroll
        for (int pos = 0; pos < 4; ++pos) {
            const uint4 sc = sv[pos * GH / 4], z = zv[pos * GH / 4];
            const float off = slot_offset<KB, true>(pos);
            *reinterpret_cast<uint4 *>(p + pos * 128) = make_uint4(
                ck_affine(unpack<KB, true>(W[0], pos), off, sc.x, z.x), ck_affine(unpack<KB, true>(W[1], pos), off, sc.y, z.y),
                ck_affine(unpack<KB, true>(W[2], pos), off, sc.z, z.z), ck_affine(unpack<KB, true>(W[3], pos), off, sc.w, z.w));
        }
    }
}
// V^^T of a record's 64 tokens, tokens in fw_tok's order (tile: the first
// chunk of 8), by one warp: a turn restores 32 channels of 32 tokens, lane
// (gq, tq) the tokens at position 8 tq of channels 8 ci + gq.  rv, rz: the
// record's value codes, scales and zeros.
template <int D, int VB, int LG>
__device__ __forceinline__ void few_values(unsigned char *tile, const unsigned char *rv, const unsigned char *rz) {
    constexpr int WL = D * VB / 64, CS = WL < 4 ? WL : 4, NWV = D * VB / 128, NGI = D >> LG, BW = D * VB / 2;
    constexpr int GH = LG >= 5 ? 1 : 2;         // groups 32 channels span
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const uint32_t *words = reinterpret_cast<const uint32_t *>(rv) + lane * CS;
    const __half *vsz = reinterpret_cast<const __half *>(rz) + 4 * tq;
    unsigned char *dst = tile + (size_t)tq * fw_vs(D) + gq * 16;
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
        const int c4 = k >> 1, vp = k & 1;      // 32 channels, two value blocks
        // the words of these channels (2 bits: half of a word), of tokens [block][p]
        const int wi = VB == 2 ? c4 >> 1 : c4, sh = VB == 2 ? (c4 & 1) * 8 : 0;
        uint32_t W[2][2];
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int u = p * NWV + wi;
                W[v][p] = words[(2 * vp + v) * BW + u / CS * 32 * CS + u % CS] >> sh;
            }
        uint2 sv[GH][2], zv[GH][2];
#pragma unroll
        for (int q = 0; q < GH; ++q)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const __half *row = vsz + (2 * vp + v) * (2 * NGI * 16) + (LG >= 5 ? (32 * c4) >> LG : 2 * c4 + q) * 16;
                sv[q][v] = *reinterpret_cast<const uint2 *>(row);
                zv[q][v] = *reinterpret_cast<const uint2 *>(row + NGI * 16);
            }
        unsigned char *p = dst + vp * (4 * fw_vs(D)) + c4 * 512;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float off = slot_offset<VB, false>(q);
            const int e = q * GH / 4;
            *reinterpret_cast<uint4 *>(p + q * 128) = make_uint4(ck_affine(unpack<VB, false>(W[0][0], q), off, sv[e][0].x, zv[e][0].x),
                                                                 ck_affine(unpack<VB, false>(W[0][1], q), off, sv[e][0].y, zv[e][0].y),
                                                                 ck_affine(unpack<VB, false>(W[1][0], q), off, sv[e][1].x, zv[e][1].x),
                                                                 ck_affine(unpack<VB, false>(W[1][1], q), off, sv[e][1].y, zv[e][1].y));
        }
    }
}
// ... by the cache's bit widths and group size
template <int D, int KB>
__device__ __forceinline__ void few_keys_g(unsigned char *tile, const unsigned char *rec, int lgG) {
    switch (lgG) {
    case 4: few_keys<D, KB, 4>(tile, rec); break;
    case 5: few_keys<D, KB, 5>(tile, rec); break;
    default: few_keys<D, KB, 6>(tile, rec); break;   // one row of scales a record from G = 64 on
    }
}
template <int D, int VB>
__device__ __forceinline__ void few_values_g(unsigned char *tile, const unsigned char *rv, const unsigned char *rz,
                                             int lgG) {
    switch (lgG) {
    case 4: few_values<D, VB, 4>(tile, rv, rz); break;
    case 5: few_values<D, VB, 5>(tile, rv, rz); break;
    case 6: few_values<D, VB, 6>(tile, rv, rz); break;
    default:
        if constexpr (D >= 128) few_values<D, VB, 7>(tile, rv, rz);
        break;
    }
}
template <int D>
__device__ __forceinline__ void few_keys(const KiviGeom &g, unsigned char *tile, const unsigned char *rec, int lgG) {
    if (g.kbits == 2) few_keys_g<D, 2>(tile, rec, lgG);
    else few_keys_g<D, 4>(tile, rec, lgG);
}
template <int D>
__device__ __forceinline__ void few_values(const KiviGeom &g, unsigned char *tile, const unsigned char *rec, int lgG) {
    if (g.vbits == 2) few_values_g<D, 2>(tile, rec + g.off_vc, rec + g.off_vsz, lgG);
    else few_values_g<D, 4>(tile, rec + g.off_vc, rec + g.off_vsz, lgG);
}
// 16 bytes of a row (channels 8 c ..) to their positions in row r of a tile
// whose chunks are STEP bytes apart
template <int STEP>
__device__ __forceinline__ void fw_put(unsigned char *tile, int r, int c, const uint4 &v) {
    const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int p = fw_chan(8 * c + 2 * k);
        *reinterpret_cast<uint32_t *>(tile + (p >> 3) * STEP + r * 16 + (p & 7) * 2) = h[k];
    }
}

// 16 bytes of token tau's fp16 row, in the window or the chunk (zero past the
// chunk; chunk0: the slice's first row in chk)
template <int D>
__device__ __forceinline__ uint4 fw_row16(const CkSeg &sg, const __half *win, int ring, const __half *chk,
                                          size_t chunk0, int tau, int c) {
    const __half *src = tau < sg.T ? win + (size_t)(tau % ring) * D : chk + (chunk0 + (tau - sg.T)) * D;
    return tau < sg.T + sg.n ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
}
// Block blk of the segment with some fp16 tokens (or past the list: then its
// keys are left and its values zeroed, as their weights are zero), by one
// warp; loads go out ahead of the stores.
template <int D>
__device__ __noinline__ void cold_keys(const KiviGeom &g, const KiviDev &dv, const __half *Kn, const ChunkArgs &a,
                                       const CkSeg &sg, int blk, unsigned char *kt, const unsigned char *rec) {
    constexpr int CPR = D / 8, U = 8;
    const int lane = threadIdx.x & 31, v = 2 * sg.x0 + blk, Tqk = a.Tqk[sg.i];
    if (v >= sg.nb) return;
    const int tb = sg.bl.phys(v) * KIVI_KBLK, r0 = max(Tqk - tb, 0);   // rows below r0 are quantized
    if (r0 > 0) few_keys<D>(g, kt, rec, __ffs(g.G) - 1);
    __syncwarp();
    const __half *win = dv.Kf + kf_slice(g, sg.i, sg.j);
    const size_t chunk0 = ((size_t)sg.i * g.h + sg.j) * a.n_stride;
    for (int e0 = r0 * CPR + lane; e0 < KIVI_KBLK * CPR; e0 += 32 * U) {
        uint4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = min(e0 + 32 * k, KIVI_KBLK * CPR - 1);
            x[k] = fw_row16<D>(sg, win, g.R, Kn, chunk0, tb + e / CPR, e % CPR);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = e0 + 32 * k;
            if (e < KIVI_KBLK * CPR) fw_put<kFwKS>(kt, e / CPR, e % CPR, x[k]);
        }
    }
}
template <int D>
__device__ __noinline__ void cold_values(const KiviGeom &g, const KiviDev &dv, const __half *Vn, const ChunkArgs &a,
                                         const CkSeg &sg, int blk, unsigned char *vt, const unsigned char *rec) {
    constexpr int CPR = D / 8, U = 8;
    const int lane = threadIdx.x & 31, v = 2 * sg.x0 + blk, Tqv = a.Tqv[sg.i];
    if (v >= sg.nb) {
        for (int e = lane; e < KIVI_KBLK / 8 * (fw_vs(D) / 16); e += 32) reinterpret_cast<uint4 *>(vt)[e] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int tb = sg.bl.phys(v) * KIVI_KBLK, r0 = max(Tqv - tb, 0);
    if (r0 > 0) few_values<D>(g, vt, rec, __ffs(g.G) - 1);
    __syncwarp();
    const __half *win = dv.Vf + vf_slice(g, sg.i, sg.j);
    const size_t chunk0 = ((size_t)sg.i * g.h + sg.j) * a.n_stride;
    // consecutive lanes take consecutive tokens
    for (int e0 = lane; e0 < KIVI_KBLK * CPR; e0 += 32 * U) {
        uint4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = e0 + 32 * k, rr = max(e & (KIVI_KBLK - 1), r0 & (KIVI_KBLK - 1));
            x[k] = fw_row16<D>(sg, win, g.R + 1, Vn, chunk0, tb + rr, e / KIVI_KBLK);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int e = e0 + 32 * k, rr = e & (KIVI_KBLK - 1), c = e / KIVI_KBLK, pos = fw_tok(rr);
            if (rr < r0) continue;
            const uint32_t h[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            unsigned char *dst = vt + (pos >> 3) * fw_vs(D) + c * 128 + (pos & 7) * 2;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint16_t *>(dst + q * 16) = (uint16_t)(h[q >> 1] >> (16 * (q & 1)));
        }
    }
}

// A raise: the rows' maxima over the tile (tS: this warp's scores; hid: does
// a row miss part of the block), the references of the rows that grew by
// more than 2^8, and their factors.  Called by every softmax warp.
__device__ __noinline__ void raise_refs(uint32_t tS, float sl2, bool cut, int key, int p0, int e0, int hg, int W, int sinks,
                                        float *s_ref, float *s_al, float (*s_red)[kFwRows]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t r[16];
    tc_ld16(tS, r);
    tc_wait_ld();
    const uint32_t h = cut ? ck_hidden16(key, p0, e0, hg, W, sinks) : 0u;
#pragma unroll
    for (int c = 0; c < kFwRows; ++c) {
        const float m = redux_max((h >> c) & 1u ? -INFINITY : __uint_as_float(r[c]) * sl2);
        if (lane == 0) s_red[warp][c] = m;
    }
    fw_sync();
    const int t = threadIdx.x;
    if (t < kFwRows) {
        const float m = fmaxf(fmaxf(s_red[0][t], s_red[1][t]), fmaxf(s_red[2][t], s_red[3][t]));
        const float old = s_ref[t];
        const bool grow = m != -INFINITY && m + old > kCkLift + kCkLag;
        s_al[t] = grow && old != kFwUnset ? ex2((kCkLift - m) - old) : 1.f;
        if (grow) s_ref[t] = kCkLift - m;
    }
    fw_sync();
}
// O^T times the rows' factors (tO: this warp's lanes)
__device__ __noinline__ void rescale_out(uint32_t tO, const float *s_al) {
    uint32_t o[16];
    tc_ld16(tO, o);
    tc_wait_ld();
#pragma unroll
    for (int c = 0; c < kFwRows; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * s_al[c]);
    tc_st16(tO, o);
    tc_wait_st();
}

// Warps 0-3: softmax (thread t: token t of the tile, tensor-memory lane t;
// channel t of O^T); then the dequantizing warps; then one warp each for
// S^T, O^T and the record copies.  Tensor memory: S^T buffers of N
// columns from 0, then O^T.  Shared memory: K^ and V^ stages, Q [N][D], P^T
// tiles [128][N], references and sums, records.
template <int D>
__global__ void __launch_bounds__(kFwThreads, 1)
    chunk_few_kernel(KiviGeom g, KiviDev dv, const __half *__restrict__ Q, const __half *__restrict__ Kn,
                     const __half *__restrict__ Vn, __half *__restrict__ O, const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int N = kFwRows, KB = fw_kb(D), VB = fw_vb(D), KS = kFwStages, PB = kFwKeys * N * 2, QB = N * D * 2;
    constexpr unsigned QLBO = N * 16, KLBO = kFwKS, VLBO = fw_vs(D);
    constexpr int BF = kFwBufs, LB = 2;             // buffers, log2 of them
    constexpr int TCOLS = 128;                      // (BF + 1) N columns, a power of two
    unsigned char *sK = smem, *sV = sK + KS * KB, *sQ = sV + KS * VB, *sP = sQ + QB, *sR = sP + BF * PB;
    // counts 4 (the softmax warps): Q, P [buffer]; 2 (a tile's two warps, a
    // record's): K and V tiles written, records read; 1: the others
    constexpr int N4 = 1 + BF, N2 = N4 + 2 * KS + kFwMaxRaw, NB = N2 + 2 * BF + 2 * KS + kFwMaxRaw;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bQ = bars, *const bP = bars + 1, *const bK = bars + N4, *const bV = bK + KS, *const eR = bV + KS,
                    *const bS = bars + N2, *const bF = bS + BF, *const eK = bF + BF, *const eV = eK + KS,
                    *const bR = eV + KS;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;
    __shared__ __align__(16) float s_ref[N];       // the lift less each row's reference (log2 units)
    __shared__ __align__(16) float s_al[N];        // a raise's rescaling factors
    __shared__ float s_red[4][N];                  // per warp: maxima, or sums
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = a.hg;
    if (tid < NB) {
        mbar_init(&bars[tid], tid < N4 ? 4 : tid < N2 ? 2 : 1);
        fence_mbar_init();
    }
    if (tid == 0) s_abort = 0;
    if (warp == 0) tc_alloc(&s_taddr, TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = s_taddr;
    const volatile int *abort = &s_abort;
    bool ok = true;
    CkWalk<> walk;
    walk.start(a, blockIdx.x);
    CkSeg sg = {};
    constexpr int WD = 4, WS = WD + 2 * kFwDq;   // first dequantizing warp, the S^T warp
    // The segment's blocks are [2 x0, nb): how many of them have a record.
    auto raw_blocks = [&](int Tq) {
        const int nb = min(2 * (sg.x0 + sg.nx), sg.nb);
        return max(0, min(nb, sg.bl.virt((Tq + KIVI_KBLK - 1) / KIVI_KBLK)) - 2 * sg.x0);
    };

    if (warp == WS) {
        // ---- S^T = K^ Q^T ----
        constexpr uint32_t ID = tc_idesc_f16(kFwKeys, N, 0);
        CkRing t;
        int cs = 0;
        unsigned qph = 0;
        const uint64_t dk = tc_desc(sK, KLBO, 128), dq = tc_desc(sQ, QLBO, 128);
        while (ok && walk.next(g, a, sg)) {
            const int nx = __reduce_max_sync(kFull, sg.nx);   // (warp-uniform)
            for (int x = 0; x < nx; ++x, ++cs, t.next(KS)) {
                // Q and K^ written, the buffer's last scores read (their P written)
                ok = (x > 0 || mbar_wait_ab(bQ, qph, abort)) && mbar_wait_ab(&bK[t.s], t.p, abort) &&
                     (cs < BF || mbar_wait_ab(&bP[cs & (BF - 1)], (unsigned)((cs >> LB) + 1) & 1u, abort));
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t d = dk + (uint32_t)(t.s * (KB >> 4));
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    tc_mma_f16_w(taddr + N * (cs & (BF - 1)), d + ((2 * c * KLBO) >> 4), dq + ((2 * c * QLBO) >> 4), ID, c > 0);
                tc_commit_w(&bS[cs & (BF - 1)]);
                tc_commit_w(&eK[t.s]);
            }
            qph ^= 1u;
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        // every commit has landed before shared memory is given up
        // (bounded; a phase already seen returns at once)
        for (int y = max(0, cs - BF); y < cs; ++y) mbar_wait(&bS[y & (BF - 1)], (unsigned)(y >> LB) & 1u);
        for (int y = max(0, cs - KS); y < cs; ++y) mbar_wait(&eK[y % KS], (unsigned)(y / KS) & 1u);
        __syncwarp();
    } else if (warp == WS + 1) {
        // ---- O^T += V^^T P^T; M 128 whatever d: with d = 64 the upper rows
        // multiply other shared memory and are not read ----
        constexpr uint32_t ID = tc_idesc_f16(128, N, 1);
        CkRing t;
        int cp = 0;
        const uint64_t dvd = tc_desc(sV, VLBO, 128), dp = tc_desc(sP, 128, kFwKeys * 16);
        while (ok && walk.next(g, a, sg)) {
            const int nx = __reduce_max_sync(kFull, sg.nx);
            for (int x = 0; x < nx; ++x, ++cp, t.next(KS)) {
                ok = mbar_wait_ab(&bV[t.s], t.p, abort) && mbar_wait_ab(&bP[cp & (BF - 1)], (unsigned)(cp >> LB) & 1u, abort);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t d = dvd + (uint32_t)(t.s * (VB >> 4)), e = dp + (uint32_t)((cp & (BF - 1)) * (PB >> 4));
#pragma unroll
                for (int c = 0; c < kFwKeys / 16; ++c)
                    tc_mma_f16_w(taddr + BF * N, d + ((2 * c * VLBO) >> 4), e + ((256 * c) >> 4), ID, x > 0 || c > 0);
                tc_commit_w(&bF[cp & (BF - 1)]);
                tc_commit_w(&eV[t.s]);
            }
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        for (int y = max(0, cp - BF); y < cp; ++y) mbar_wait(&bF[y & (BF - 1)], (unsigned)(y >> LB) & 1u);
        for (int y = max(0, cp - KS); y < cp; ++y) mbar_wait(&eV[y % KS], (unsigned)(y / KS) & 1u);
        __syncwarp();
    } else if (warp == WS + 2) {
        // ---- records (lane 0 issues) ----
        CkRing r;
        int issued = 0;
        while (walk.next(g, a, sg)) {
            if (lane == 0) {
                const int n = raw_blocks(max(a.Tqk[sg.i], a.Tqv[sg.i]));
                const unsigned char *recs = dv.blk + rec_off(g, sg.i, sg.j, 0);
                for (int y = 0; y < n; ++y, ++issued, r.next(a.rs)) {
                    ok = (issued < a.rs || mbar_wait_ab(&eR[r.s], r.p ^ 1u, abort)) && issued < a.quit;
                    if (!ok) break;
                    mbar_expect_tx(&bR[r.s], (unsigned)g.rec_bytes);
                    bulk_g2s(sR + (size_t)r.s * g.rec_bytes, recs + (size_t)sg.bl.phys(2 * sg.x0 + y) * g.rec_bytes,
                             (unsigned)g.rec_bytes, &bR[r.s]);
                }
            }
            ok = __all_sync(kFull, ok);
            if (!ok) break;
        }
        if (lane == 0) {
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            for (int y = max(0, issued - a.rs); y < issued; ++y) mbar_wait(&bR[y % a.rs], (unsigned)(y / a.rs) & 1u);
        }
        __syncwarp();
    } else if (warp >= WD) {
        // ---- K^ (the first four warps) or V^^T (the others): the CTA's blocks,
        // two a tile, in turn ----
        const int w = (warp - WD) % kFwDq, lgG = __ffs(g.G) - 1;
        const bool keys = warp < WD + kFwDq;
        uint64_t *const bT = keys ? bK : bV, *const eT = keys ? eK : eV;   // the tile written, read
        int tiles = 0;   // of the CTA so far
        CkRing seg;      // the segment's first record's stage
        while (ok && walk.next(g, a, sg)) {
            const int nraw = raw_blocks(max(a.Tqk[sg.i], a.Tqv[sg.i]));
            const int npk = sg.bl.virt(min(a.Tqk[sg.i], a.Tqv[sg.i]) / KIVI_KBLK) - 2 * sg.x0;   // fully quantized blocks
            int blk = (w - 2 * tiles) & (kFwDq - 1);   // the segment's first block of this warp
            CkRing r = seg;
            r.skip(blk, a.rs);
            for (; blk < 2 * sg.nx; blk += kFwDq, r.skip(kFwDq, a.rs)) {
                const int y = tiles + (blk >> 1), st = y % KS, half = blk & 1;
                const bool raw = blk < nraw;
                const unsigned char *rp = sR + (size_t)r.s * g.rec_bytes;
                ok = (y < KS || mbar_wait_ab(&eT[st], (unsigned)(y / KS + 1) & 1u, abort)) &&
                     (!raw || mbar_wait_ab(&bR[r.s], r.p, abort));
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                if (keys) {
                    unsigned char *kt = sK + st * KB + half * KIVI_KBLK * 16;
                    if (blk < npk) few_keys<D>(g, kt, rp, lgG);
                    else cold_keys<D>(g, dv, Kn, a, sg, blk, kt, rp);
                } else {
                    unsigned char *vt = sV + st * VB + half * (KIVI_KBLK / 8) * (int)VLBO;
                    if (blk < npk) few_values<D>(g, vt, rp, lgG);
                    else cold_values<D>(g, dv, Vn, a, sg, blk, vt, rp);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bT[st]);
                    if (raw) mbar_arrive(&eR[r.s]);
                }
            }
            tiles += sg.nx;
            seg.skip(nraw, a.rs);
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        __syncwarp();
    } else {
        // ---- the softmax warps ----
        const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
        const uint32_t tO = taddr + lane_off + BF * N;
        const float sl2 = 1.4426950408889634f / sqrtf((float)D);   // log2(e) / sqrt(d)
        const int W = a.vis.window, sinks = a.vis.sinks;
        const int kpos = fw_tok(tid);
        int cnt = 0;             // tiles so far
        while (walk.next(g, a, sg)) {
            // Q: row (r, e) from head e of token r; rows past the chunk are zero
            // (the last segment's scores are all read)
            for (int e = tid; e < N * (D / 8); e += 128) {
                const int q = e % N, c = e / N;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (sg.row0 + q < sg.nrows) {
                    const int rw = sg.row0 + q, tok = chunk_div(a, rw);
                    v = *reinterpret_cast<const uint4 *>(
                        Q + (((size_t)sg.i * a.hq + sg.j * hg + rw - tok * hg) * a.n_stride + tok) * D + 8 * c);
                }
                fw_put<N * 16>(sQ, q, c, v);
            }
            if (tid < N) s_ref[tid] = kFwUnset;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bQ);
            fw_sync();   // the references are set
            const int p0 = sg.T + chunk_div(a, sg.row0), e0 = sg.row0 - chunk_div(a, sg.row0) * hg;   // the first row's position and head
            const int p1 = sg.T + chunk_div(a, sg.nrows - 1);
            float lsum[N];
#pragma unroll
            for (int c = 0; c < N; ++c) lsum[c] = 0.f;
            for (int x = 0; x < sg.nx; ++x, ++cnt) {
                const int b = cnt & (BF - 1), v = 2 * (sg.x0 + x) + (tid >> 6);
                const int kb = v < sg.nb ? sg.bl.phys(v) * KIVI_KBLK : 0x7fffff00, key = kb + (tid & 63);
                const uint32_t tS = taddr + lane_off + N * b;
                ok = ok && __all_sync(kFull, mbar_wait_ab(&bS[b], (unsigned)(cnt >> LB) & 1u, abort));
                tc_fence_after();
                // some row does not see all of this warp's block
                const bool cut = kb + KIVI_KBLK - 1 > p0 || (W > 0 && kb <= p1 - W && kb + KIVI_KBLK > sinks);
                // the scores of this token as log2 weights against the rows'
                // references, masked
                auto scores = [&](float (&y)[N]) {
                    uint32_t r[N];
                    tc_ld16(tS, r);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < N; c += 4) {
                        const float4 ref = *reinterpret_cast<const float4 *>(s_ref + c);
                        y[c] = fmaf(__uint_as_float(r[c]), sl2, ref.x);
                        y[c + 1] = fmaf(__uint_as_float(r[c + 1]), sl2, ref.y);
                        y[c + 2] = fmaf(__uint_as_float(r[c + 2]), sl2, ref.z);
                        y[c + 3] = fmaf(__uint_as_float(r[c + 3]), sl2, ref.w);
                    }
                    if (cut) {
                        const uint32_t h = ck_hidden16(key, p0, e0, hg, W, sinks);
#pragma unroll
                        for (int c = 0; c < N; ++c)
                            if ((h >> c) & 1u) y[c] = -INFINITY;
                    }
                };
                float s[N], up = -INFINITY;   // the largest lifted log2 weight
                if (ok) {
                    scores(s);
#pragma unroll
                    for (int c = 0; c < N; ++c) up = fmaxf(up, s[c]);
                }
                const bool raise = fw_any(!ok || up > kCkLift + kCkLag);
                if (raise) {
                    // every warp learns whether one has given up
                    if (fw_any(!ok)) {
                        ok = false;
                        break;
                    }
                    raise_refs(tS, sl2, cut, key, p0, e0, hg, W, sinks, s_ref, s_al, s_red);
#pragma unroll
                    for (int c = 0; c < N; ++c) lsum[c] *= s_al[c];
                    if (x > 0) {   // O^T, once O^T of tile x - 1 is in
                        ok = __all_sync(kFull, mbar_wait_ab(&bF[(cnt - 1) & (BF - 1)], (unsigned)((cnt - 1) >> LB) & 1u, abort));
                        if (ok) {
                            tc_fence_after();
                            rescale_out(tO, s_al);
                        }
                    }
                }
                // P^T: this buffer's last O^T has read its weights
                if (ok && cnt >= BF) ok = __all_sync(kFull, mbar_wait_ab(&bF[b], (unsigned)((cnt >> LB) + 1) & 1u, abort));
                if (!ok) continue;   // the next vote ends it for every warp
                if (raise) scores(s);   // against the new references
                uint32_t pw[N / 2];
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    const float y0 = ex2(s[c]), y1 = ex2(s[c + 1]);
                    lsum[c] += y0;
                    lsum[c + 1] += y1;
                    pw[c / 2] = ck_pack(y0, y1);
                }
#pragma unroll
                for (int k = 0; k < N / 8; ++k)
                    *reinterpret_cast<uint4 *>(sP + b * PB + (k * kFwKeys + kpos) * 16) =
                        make_uint4(pw[4 * k], pw[4 * k + 1], pw[4 * k + 2], pw[4 * k + 3]);
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bP[b]);
            }
            for (int y = max(cnt - BF, 0); y < cnt && ok; ++y)
                ok = __all_sync(kFull, mbar_wait_ab(&bF[y & (BF - 1)], (unsigned)(y >> LB) & 1u, abort));
            if (fw_any(!ok)) {   // for every warp
                ok = false;
                break;
            }
            tc_fence_after();
            // the rows' sums over the threads
#pragma unroll
            for (int c = 0; c < N; ++c) {
                float l = lsum[c];
#pragma unroll
                for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
                if (lane == 0) s_red[warp][c] = l;
            }
            fw_sync();
            // O^T to rows of D floats (the P^T buffers are free), then a row a warp
            float *rows = reinterpret_cast<float *>(sP);
            static_assert((size_t)N * D * 4 <= (size_t)BF * PB, "the rows fit");
            uint32_t o[N];
            tc_ld16(tO, o);
            tc_wait_ld();
            if (tid < D)
#pragma unroll
                for (int c = 0; c < N; ++c) rows[c * D + tid] = __uint_as_float(o[c]);
            fw_sync();
            const bool part = sg.nx < sg.nt;
            const size_t pr = (size_t)(2 * blockIdx.x + (sg.x0 == 0 ? 1 : 0)) * N;
#pragma unroll 1
            for (int q = warp; q < min(sg.nrows - sg.row0, N); q += 4) {
                constexpr int V = D / 32;
                const float l = s_red[0][q] + s_red[1][q] + s_red[2][q] + s_red[3][q];
                float v[V];
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = rows[q * D + lane * V + k];
                if (part) {
                    if (lane == 0)
                        reinterpret_cast<float2 *>(a.ml)[pr + q] = make_float2(s_ref[q] == kFwUnset ? -INFINITY : -s_ref[q], l);
                    float *dst = a.acc + (pr + q) * D + lane * V;
#pragma unroll
                    for (int k = 0; k < V; k += 2) *reinterpret_cast<float2 *>(dst + k) = make_float2(v[k], v[k + 1]);
                } else {
                    const float inv = 1.f / l;
                    const int rw = sg.row0 + q, tok = chunk_div(a, rw);
                    __half *dst = O + (((size_t)sg.i * a.hq + sg.j * hg + rw - tok * hg) * a.n_stride + tok) * D + lane * V;
#pragma unroll
                    for (int k = 0; k < V; k += 2) *reinterpret_cast<uint32_t *>(dst + k) = ck_pack(v[k] * inv, v[k + 1] * inv);
                }
            }
            tc_fence_before();
            fw_sync();   // the sums are read
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(taddr, TCOLS);
}

}  // namespace
