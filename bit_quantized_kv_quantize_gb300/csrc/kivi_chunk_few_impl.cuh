// kivi_chunk_few_impl.cuh -- chunk attention where each kv head has few query
// rows (a speculative step's tokens, a short last piece): the transposed form
// of the chunk attention (kivi_chunk_attn_impl.cuh has the mathematics).
//
// With 128 query rows on the MMA's M side, a few rows leave most of the tensor
// cores' and the softmax's work padding, and a tile takes about 1800 cycles
// however few the rows.  Here the tokens are on the M side and the rows on N
// (N = 16, 32 or 64):
//   S^T [128 tokens x N] = K^ Q^T,   O^T [d x N] += V^^T P^T,
// so a tile of 128 tokens costs 16 MMAs of N columns, thread t of the softmax
// owns token t and computes N weights, and what remains is restoring the
// tile: the kernel is bound by the dequantizing warps' instructions (4.5 a
// pair of values) and by HBM.
//
// The softmax needs a row's maximum over the tile's tokens, which are spread
// over the threads.  It is not formed a tile: the weights are taken against
// the row's reference, and only when some score lies more than 2^8 above it
// (one vote of the four warps a tile) are the maxima formed (redux.f32 over
// the lanes, then the warps), the references raised, and O^T and the sums
// rescaled.  A thread keeps its own part of each row's sum; they are added up
// at the end of the segment.
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

constexpr int kFwKeys = 128;    // tokens of a tile (two blocks)
constexpr int kFwStages = 2;    // K^ tiles, and V^ tiles, in flight
constexpr int kFwMaxRaw = 12;   // records in flight
// Dequantizing groups.  Four of them where the softmax warps' registers allow
// it (80 a thread), else two (128): one group alone restores a block in about
// 1200 cycles.
__host__ __device__ constexpr int fw_groups(int N) { return N == 16 ? 4 : 2; }
__host__ __device__ constexpr int fw_threads(int N) { return 32 * (4 + fw_groups(N) * kCkDqGroup + 3); }
// S^T and P^T buffers: tiles that the softmax may be apart from either MMA
// (four hide the waits between the roles; with 64 rows there is room for two)
__host__ __device__ constexpr int fw_bufs(int N) { return N == 64 ? 2 : 4; }
constexpr float kFwUnset = 1e30f;   // minus the reference of a row that has seen nothing

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

// A dequantizing group's state.
struct FwGroup {
    int w, dt, lgG, meets;   // warp, thread of the group; log2 G; meetings so far
    uint64_t *bX;
    const volatile int *abort;
    // the group's warps meet (a bounded wait, unlike a named barrier)
    __device__ __forceinline__ bool meet() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bX);
        return __all_sync(kFull, mbar_wait_ab(bX, (unsigned)meets++ & 1u, abort)) != 0;
    }
};
// 16 bytes of token tau's fp16 row, in the window or the chunk (zero past the
// chunk; chunk0: the slice's first row in chk)
template <int D>
__device__ __forceinline__ uint4 fw_row16(const CkSeg &sg, const __half *win, int ring, const __half *chk,
                                          size_t chunk0, int tau, int c) {
    const __half *src = tau < sg.T ? win + (size_t)(tau % ring) * D : chk + (chunk0 + (tau - sg.T)) * D;
    return tau < sg.T + sg.n ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
}
// Block blk of the segment with some fp16 tokens (or past the list: then its
// keys are left and its values zeroed, as their weights are zero).  False if
// a wait ran out.
template <int D>
__device__ __noinline__ bool cold_keys(FwGroup &f, const KiviGeom &g, const KiviDev &dv, const __half *Kn,
                                       const ChunkArgs &a, const CkSeg &sg, int blk, unsigned char *kt,
                                       const unsigned char *rec) {
    constexpr int CPR = D / 8;
    const int v = 2 * sg.x0 + blk, Tqk = a.Tqk[sg.i];
    if (v >= sg.nb) return true;
    const int tb = sg.bl.phys(v) * KIVI_KBLK, r0 = max(Tqk - tb, 0);   // rows below r0 are quantized
    if (r0 > 0) dequant_keys_cold<D, kFwKeys>(kt, rec, g.kbits, g.off_ksz, f.lgG, f.w);
    if (r0 >= KIVI_KBLK) return true;
    if (r0 > 0 && !f.meet()) return false;
    const __half *win = dv.Kf + kf_slice(g, sg.i, sg.j);
    const size_t chunk0 = ((size_t)sg.i * g.h + sg.j) * a.n_stride;
    for (int e = f.dt; e < (KIVI_KBLK - r0) * CPR; e += 32 * kCkDqGroup) {
        const int rr = r0 + e / CPR, c = e % CPR;
        *reinterpret_cast<uint4 *>(kt + c * (kFwKeys * 16) + rr * 16) = fw_row16<D>(sg, win, g.R, Kn, chunk0, tb + rr, c);
    }
    return true;
}
template <int D>
__device__ __noinline__ bool cold_values(FwGroup &f, const KiviGeom &g, const KiviDev &dv, const __half *Vn,
                                         const ChunkArgs &a, const CkSeg &sg, int blk, unsigned char *vt,
                                         const unsigned char *rec) {
    constexpr int CPR = D / 8;
    const int v = 2 * sg.x0 + blk, Tqv = a.Tqv[sg.i];
    if (v >= sg.nb) {
        for (int e = f.dt; e < KIVI_KBLK / 8 * D; e += 32 * kCkDqGroup)
            reinterpret_cast<uint4 *>(vt)[e] = make_uint4(0u, 0u, 0u, 0u);
        return true;
    }
    const int tb = sg.bl.phys(v) * KIVI_KBLK, r0 = max(Tqv - tb, 0);
    if (r0 > 0) dequant_values_cold<D>(vt, rec, g.vbits, g.off_vc, g.off_vsz, f.lgG, f.w);
    if (r0 >= KIVI_KBLK) return true;
    if (r0 > 0 && !f.meet()) return false;
    const __half *win = dv.Vf + vf_slice(g, sg.i, sg.j);
    const size_t chunk0 = ((size_t)sg.i * g.h + sg.j) * a.n_stride;
    const int nr = KIVI_KBLK - r0;
    for (int e = f.dt; e < nr * CPR; e += 32 * kCkDqGroup) {
        // consecutive lanes take consecutive tokens
        const int rr = r0 + e % nr, c = e / nr;
        const uint4 u = fw_row16<D>(sg, win, g.R + 1, Vn, chunk0, tb + rr, c);
        const uint32_t h[4] = {u.x, u.y, u.z, u.w};
        unsigned char *dst = vt + (rr >> 3) * (D * 16) + c * 128 + (rr & 7) * 2;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint16_t *>(dst + k * 16) = (uint16_t)(h[k >> 1] >> (16 * (k & 1)));
    }
    return true;
}

// A raise: the rows' maxima over the tile (tS: this warp's scores; hid: does
// a row miss part of the block), the references of the rows that grew by
// more than 2^8, and their factors.  Called by every softmax warp.
template <int N>
__device__ __noinline__ void raise_refs(uint32_t tS, float sl2, bool cut, int key, int p0, int e0, int hg, int W, int sinks,
                                        float *s_ref, float *s_al, float (*s_red)[N]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int c0 = 0; c0 < N; c0 += 16) {
        uint32_t r[16];
        tc_ld16(tS + c0, r);
        tc_wait_ld();
        const uint32_t h = cut ? ck_hidden16(key, c0, p0, e0, hg, W, sinks) : 0u;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const float m = redux_max((h >> c) & 1u ? -INFINITY : __uint_as_float(r[c]) * sl2);
            if (lane == 0) s_red[warp][c0 + c] = m;
        }
    }
    fw_sync();
    const int t = threadIdx.x;
    if (t < N) {
        const float m = fmaxf(fmaxf(s_red[0][t], s_red[1][t]), fmaxf(s_red[2][t], s_red[3][t]));
        const float old = s_ref[t];
        const bool grow = m != -INFINITY && m + old > 8.f;
        s_al[t] = grow && old != kFwUnset ? ex2(-old - m) : 1.f;
        if (grow) s_ref[t] = -m;
    }
    fw_sync();
}
// O^T times the rows' factors (tO: this warp's lanes)
template <int N>
__device__ __noinline__ void rescale_out(uint32_t tO, const float *s_al) {
#pragma unroll 1
    for (int c0 = 0; c0 < N; c0 += 16) {
        uint32_t o[16];
        tc_ld16(tO + c0, o);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * s_al[c0 + c]);
        tc_st16(tO + c0, o);
    }
    tc_wait_st();
}

// Warps 0-3: softmax (thread t: token t of the tile, tensor-memory lane t;
// channel t of O^T); then the dequantizing groups; then one warp each for
// S^T, O^T and the record copies.  Tensor memory: S^T buffers of N
// columns from 0, then O^T.  Shared memory: K^ and V^ stages, Q [N][D], P^T
// tiles [128][N], references and sums, records.
template <int D, int N>
__global__ void __launch_bounds__(fw_threads(N), 1)
    chunk_few_kernel(KiviGeom g, KiviDev dv, const __half *__restrict__ Q, const __half *__restrict__ Kn,
                     const __half *__restrict__ Vn, __half *__restrict__ O, const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int G = fw_groups(N), TB = kFwKeys * D * 2, KS = kFwStages, PB = kFwKeys * N * 2, QB = N * D * 2;
    constexpr unsigned QLBO = N * 16, KLBO = kFwKeys * 16, VLBO = D * 16;
    constexpr int BF = fw_bufs(N), TCOLS = N == 16 ? 128 : 256;   // (BF + 1) N columns, a power of two
    constexpr int LB = BF == 4 ? 2 : 1;                           // log2 of the buffers
    unsigned char *sK = smem, *sV = sK + KS * TB, *sQ = sV + KS * TB, *sP = sQ + QB, *sR = sP + BF * PB;
    // counts 8 (two groups): K and V tiles written; 4: Q, P [buffer], the
    // groups' meetings, records read; 1: the others
    constexpr int N8 = 2 * KS, N4 = N8 + 1 + BF + G + kFwMaxRaw, NB = N4 + 2 * BF + 2 * KS + kFwMaxRaw;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bK = bars, *const bV = bK + KS, *const bQ = bars + N8, *const bP = bQ + 1, *const bX = bP + BF,
                    *const eR = bX + G, *const bS = bars + N4, *const bF = bS + BF, *const eK = bF + BF,
                    *const eV = eK + KS, *const bR = eV + KS;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;
    __shared__ __align__(16) float s_ref[N];       // minus each row's reference (log2 units)
    __shared__ __align__(16) float s_al[N];        // a raise's rescaling factors
    __shared__ float s_red[4][N];                  // per warp: maxima, or sums
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = a.hg;
    if (tid < NB) {
        mbar_init(&bars[tid], tid < N8 ? 8 : tid < N4 ? 4 : 1);
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
    CkWalk walk;
    walk.start(a, blockIdx.x);
    CkSeg sg = {};
    constexpr int WD = 4, WS = WD + G * kCkDqGroup;   // first dequantizing warp, the S^T warp
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
                const uint64_t d = dk + (uint32_t)(t.s * (TB >> 4));
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
                const uint64_t d = dvd + (uint32_t)(t.s * (TB >> 4)), e = dp + (uint32_t)((cp & (BF - 1)) * (PB >> 4));
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
                    ok = issued < a.rs || mbar_wait_ab(&eR[r.s], r.p ^ 1u, abort);
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
        // ---- K^ and V^^T: the CTA's tile y is restored by groups 2 y mod G
        // and 2 y + 1 mod G, a block each ----
        const int grp = (warp - WD) / kCkDqGroup, half = grp & 1;
        FwGroup f;
        f.w = (warp - WD) % kCkDqGroup;
        f.dt = (tid - 32 * WD) & (32 * kCkDqGroup - 1);
        f.lgG = __ffs(g.G) - 1;
        f.meets = 0;
        f.bX = &bX[grp];
        f.abort = abort;
        int tiles = 0, recs = 0;   // of the CTA so far
        while (ok && walk.next(g, a, sg)) {
            const int nraw = raw_blocks(max(a.Tqk[sg.i], a.Tqv[sg.i]));
            const int npk = sg.bl.virt(min(a.Tqk[sg.i], a.Tqv[sg.i]) / KIVI_KBLK) - 2 * sg.x0;   // fully quantized blocks
            // the segment's first tile of this group; its stage, and the
            // record's (if any)
            int x = ((grp >> 1) - tiles % (G / 2) + G / 2) % (G / 2);
            for (; x < sg.nx; x += G / 2) {
                const int y = tiles + x, st = y % KS, blk = 2 * x + half, rec = recs + blk, rst = rec % a.rs;
                const unsigned tp = (unsigned)(y / KS) & 1u;
                const bool raw = blk < nraw;
                unsigned char *kt = sK + st * TB + half * KIVI_KBLK * 16;
                unsigned char *vt = sV + st * TB + half * (KIVI_KBLK / 8) * (int)VLBO;
                const unsigned char *rp = sR + (size_t)rst * g.rec_bytes;
                ok = (y < KS || mbar_wait_ab(&eK[st], tp ^ 1u, abort)) &&
                     (!raw || mbar_wait_ab(&bR[rst], (unsigned)(rec / a.rs) & 1u, abort));
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                if (blk < npk) {
                    if (g.kbits == 2) dequant_keys<D, 2, kFwKeys>(kt, rp, g.off_ksz, f.lgG, f.w);
                    else dequant_keys<D, 4, kFwKeys>(kt, rp, g.off_ksz, f.lgG, f.w);
                } else if (!(ok = cold_keys<D>(f, g, dv, Kn, a, sg, blk, kt, rp))) {
                    break;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bK[st]);
                ok = __all_sync(kFull, y < KS || mbar_wait_ab(&eV[st], tp ^ 1u, abort));
                if (!ok) break;
                if (blk < npk) {
                    if (g.vbits == 2) dequant_values<D, 2>(vt, rp, g.off_vc, g.off_vsz, f.lgG, f.w);
                    else dequant_values<D, 4>(vt, rp, g.off_vc, g.off_vsz, f.lgG, f.w);
                } else if (!(ok = cold_values<D>(f, g, dv, Vn, a, sg, blk, vt, rp))) {
                    break;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bV[st]);
                    if (raw) mbar_arrive(&eR[rst]);
                }
            }
            tiles += sg.nx;
            recs += nraw;
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
        constexpr int CH = 16;   // columns at a time
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
                *reinterpret_cast<uint4 *>(sQ + c * QLBO + q * 16) = v;
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
                const int kb = v < sg.nb ? sg.bl.phys(v) * KIVI_KBLK : 1 << 30, key = kb + (tid & 63);
                const uint32_t tS = taddr + lane_off + N * b;
                ok = ok && __all_sync(kFull, mbar_wait_ab(&bS[b], (unsigned)(cnt >> LB) & 1u, abort));
                tc_fence_after();
                // some row does not see all of this warp's block
                const bool cut = kb + KIVI_KBLK - 1 > p0 || (W > 0 && kb <= p1 - W && kb + KIVI_KBLK > sinks);
                // 16 scores of this token in log2 units, masked
                auto scores = [&](int c0, float (&s)[CH]) {
                    uint32_t r[CH];
                    tc_ld16(tS + c0, r);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < CH; ++c) s[c] = __uint_as_float(r[c]) * sl2;
                    if (cut) {
                        const uint32_t h = ck_hidden16(key, c0, p0, e0, hg, W, sinks);
#pragma unroll
                        for (int c = 0; c < CH; ++c)
                            if ((h >> c) & 1u) s[c] = -INFINITY;
                    }
                };
                float s[CH], up = -INFINITY;   // the most that a score lies above its reference
                if (ok)
#pragma unroll
                    for (int c0 = 0; c0 < N; c0 += CH) {
                        scores(c0, s);
#pragma unroll
                        for (int c = 0; c < CH; ++c) up = fmaxf(up, s[c] + s_ref[c0 + c]);
                    }
                const bool raise = fw_any(!ok || up > 8.f);
                if (raise) {
                    // every warp learns whether one has given up
                    if (fw_any(!ok)) {
                        ok = false;
                        break;
                    }
                    raise_refs<N>(tS, sl2, cut, key, p0, e0, hg, W, sinks, s_ref, s_al, s_red);
#pragma unroll
                    for (int c = 0; c < N; ++c) lsum[c] *= s_al[c];
                    if (x > 0) {   // O^T, once O^T of tile x - 1 is in
                        ok = __all_sync(kFull, mbar_wait_ab(&bF[(cnt - 1) & (BF - 1)], (unsigned)((cnt - 1) >> LB) & 1u, abort));
                        if (ok) {
                            tc_fence_after();
                            rescale_out<N>(tO, s_al);
                        }
                    }
                }
                // P^T: this buffer's last O^T has read its weights
                if (ok && cnt >= BF) ok = __all_sync(kFull, mbar_wait_ab(&bF[b], (unsigned)((cnt >> LB) + 1) & 1u, abort));
                if (!ok) continue;   // the next vote ends it for every warp
#pragma unroll
                for (int c0 = 0; c0 < N; c0 += CH) {
                    if (N > CH || raise) scores(c0, s);   // (one group of columns: still there)
                    uint32_t pw[CH / 2];
#pragma unroll
                    for (int c = 0; c < CH; c += 2) {
                        const float y0 = ex2(s[c] + s_ref[c0 + c]), y1 = ex2(s[c + 1] + s_ref[c0 + c + 1]);
                        lsum[c0 + c] += y0;
                        lsum[c0 + c + 1] += y1;
                        pw[c / 2] = ck_pack(y0, y1);
                    }
#pragma unroll
                    for (int k = 0; k < CH / 8; ++k)
                        *reinterpret_cast<uint4 *>(sP + b * PB + ((c0 / 8 + k) * kFwKeys + tid) * 16) =
                            make_uint4(pw[4 * k], pw[4 * k + 1], pw[4 * k + 2], pw[4 * k + 3]);
                }
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
#pragma unroll
            for (int c0 = 0; c0 < N; c0 += CH) {
                uint32_t o[CH];
                tc_ld16(tO + c0, o);
                tc_wait_ld();
                if (tid < D)
#pragma unroll
                    for (int c = 0; c < CH; ++c) rows[(c0 + c) * D + tid] = __uint_as_float(o[c]);
            }
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
