// kivi_chunk_attn_impl.cuh -- attention of a chunk of new tokens over the
// quantized cache and the chunk itself, on the 5th-generation tensor cores.
//
// Mathematics.  Row (r, e) of kv head j is query head j hg + e of chunk token
// r, at position p = T + r:
//   out = sum_s softmax_s(q . K^_s / sqrt(d)) V^_s   over the visible s <= p,
// K^_s = scale code + zero for the quantized tokens ("Literature audit --
// Group 2", section 1 KIVI, core algorithm item 5), the fp16 rows for the
// window's and the chunk's.  All hg heads of a kv head share its tokens, so
// the rows (r, e) are one list, row index r hg + e, cut into row tiles of
// 256 (two slots of 128).  A prompt's windowed attention is the same with
// nothing cached (T = 0).
//
// Per 64-token block the CTA restores K^ and V^ once as fp16 tiles in shared
// memory (dequantizing warps), S = Q K^T and O += P V run on tcgen05 with
// S, P and O in tensor memory and one thread a row doing the online softmax.
// K^ and V^ round once to fp16 (2^-11 relative a value, as the weights P
// do): the two-term operands that the one-token decode uses would double the
// MMAs, and the errors of the rounded values are independent, so they
// average like the values themselves (relative L2 error 3.6e-4 on even keys,
// 5e-4 to 1.2e-3 where keys have channels 8 times the others; an fp16 output
// alone rounds by 2.1e-4).
//
// Bound: the tensor cores, where the rows are many.  A tile's MMAs take 1280
// cycles (M 128 x N 64 x K 16 from shared memory 49, N 128 from tensor memory
// 65); the loop takes 2000 without the restoring and 2250 with it: the
// dequantizing warps' stores and the MMAs' operand reads share shared memory.
// Measured: 2048 tokens of 32 / 8 heads over 16.5k 2-bit tokens 515 us (1.14
// PFLOP/s; 303 us at the cuBLAS rate), 200 tokens 93 us, 16 tokens of 8
// sequences over 32k 215 us; a prompt of 8191 tokens, window 2048, 32 / 8
// heads, 279 us beside 32 us of packing, one of 4096, window 1024, 32 heads,
// 116 beside 45.
//
// Pipeline.  A slot has one S buffer of 64 columns, two P buffers of 32 and O.
// The scores are read into registers at once, so S of the next tile runs
// under the softmax of this one, and P V of the last tile too.  (With P
// written over its scores in one of two S buffers, S of a tile had to wait for
// P V of the last but one: 1100 cycles of softmax a tile and 600 of waiting
// for scores, measured.)  A warp issues a slot's S MMAs, another both slots'
// P V MMAs, so that a wait of one does not hold the others back.
//
// Records (packed codes, scales, zeros) come into a ring of shared-memory
// stages, one bulk copy each, several ahead.  Four warps restore a tile: K^
// as rows of tokens, V^ as rows of channels (transposed: the value words hold
// two tokens of one channel, so each half2 they yield is contiguous along
// tokens); both stores are free of bank conflicts, and the MMA's descriptor
// takes V^ K-major.  Whole tiles of chunk tokens come by TMA; other fp16
// tokens (the windows, a ragged end) are copied as rows.  V rows are taken
// MN-major.
//
// Work split (persistent, one CTA an SM): the tiles of all row tiles are laid
// end to end, each row tile led by kCkLead units that stand for its fixed
// cost, and CTA c takes an equal contiguous share.  A row tile that several
// CTAs share leaves unnormalized partials (max, sum, O), joined by a second
// kernel.
#pragma once
#include <climits>

#include "kivi_chunk_tiles.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_tma.cuh"

namespace {

constexpr int kCkRows = 128;     // rows of a slot
constexpr int kCkTileRows = 2 * kCkRows;
constexpr int kCkKeys = KIVI_KBLK;   // tokens of a tile
constexpr int kCkStages = 3;     // K^ tiles, and V^ tiles, in flight
constexpr int kCkMaxRaw = 8;     // records in flight
// Dequantizing warps: all that 16 warps of 128 registers leave.  (Eight, at 96
// to 112 registers for the softmax, took 616 to 660 us where four took 545;
// two for K^ and two for V^, a tile a warp, 600.)
constexpr int kCkDq = kCkDqGroup;
constexpr int kCkOut = 8 * 32 * 64;   // a softmax warp's 32 rows x 32 columns of the output
constexpr int kCkThreads = 32 * (8 + kCkDq + 4);

// {a, b} as one 64-bit operand of the packed fp32 instructions
__device__ __forceinline__ unsigned long long ck_f2(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void ck_f2(unsigned long long v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long ck_fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long ck_add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// One dequantizing warp's share of n tiles, all fully quantized: the loop that
// most of a long cache runs in, kept apart (and short) from the tiles with
// fp16 tokens.  t: the tile stages' position (tiles: tiles so far), r: the
// record stages'.  False if a wait ran out.
template <int D, int KB, int VB>
__device__ __forceinline__ bool packed_tiles(int n, int &tiles, CkRing &t, CkRing &r, unsigned char *sK,
                                             unsigned char *sV, const unsigned char *sR, const KiviGeom &g, int rs,
                                             int w, uint64_t *bK, uint64_t *eK, uint64_t *bV, uint64_t *eV,
                                             uint64_t *bR, uint64_t *eR, const volatile int *abort) {
    constexpr int TB = kCkKeys * D * 2;
    const int lane = threadIdx.x & 31, lgG = __ffs(g.G) - 1;
    bool rk = false, rr = false;   // polled ahead: the K stage is free, the record is in
    for (int x = 0; x < n; ++x, ++tiles) {
        bool ok = (rk || tiles < kCkStages || mbar_wait_ab(&eK[t.s], t.p ^ 1u, abort)) &&
                  (rr || mbar_wait_ab(&bR[r.s], r.p, abort));
        if (!__all_sync(kFull, ok)) return false;
        const bool rv = tiles < kCkStages || mbar_test(&eV[t.s], t.p ^ 1u);   // (seen after the keys)
        const unsigned char *rec = sR + (size_t)r.s * g.rec_bytes;
        dequant_keys<D, KB, kCkKeys>(sK + t.s * TB, rec, g.off_ksz, lgG, w);
        ok = rv || mbar_wait_ab(&eV[t.s], t.p ^ 1u, abort);
        if (!__all_sync(kFull, ok)) return false;
        CkRing t1 = t, r1 = r;
        t1.next(kCkStages);
        r1.next(rs);
        rk = x + 1 < n && tiles + 1 >= kCkStages && mbar_test(&eK[t1.s], t1.p ^ 1u);
        rr = x + 1 < n && mbar_test(&bR[r1.s], r1.p);
        dequant_values<D, VB>(sV + t.s * TB, rec, g.off_vc, g.off_vsz, lgG, w);
        // (one fence for both: telling of K^ before V^ is written takes longer,
        // 514 against 502 us for 2048 tokens over 16.5k)
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bK[t.s]);
            mbar_arrive(&bV[t.s]);
            mbar_arrive(&eR[r.s]);
        }
        t = t1;
        r = r1;
    }
    return true;
}

// After a wait ran out: the copies of chunk tiles that this thread (the first
// dequantizing warp's) asked for have landed before shared memory is given up
// (bounded).  Those of its last KS tiles may not have been waited for; they
// complete the phases of tiles written, in place of the warps that stopped
// before them (put: the warps' arrivals at bK, and at bV).
template <int KS>
__device__ __noinline__ void drain_tiles(const int (*put)[kCkDq], uint64_t *bK, uint64_t *bV) {
    for (int k = 0; k < 2; ++k) {
        uint64_t *const bT = k ? bV : bK;
        for (int y = max(0, put[k][0] - KS); y < put[k][0]; ++y) {
            for (int w = 1; w < kCkDq; ++w)
                if (put[k][w] <= y) mbar_arrive(&bT[y % KS]);
            mbar_wait(&bT[y % KS], (unsigned)(y / KS) & 1u);
        }
    }
}

// One TMA copy of 128 rows of Q into dst (chunk-major): rows (r, e), e fastest,
// from token r0 on, of (sequence, kv head) bh.
__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *tm, int r0, int bh, uint64_t *bar,
                                         unsigned bytes) {
    mbar_expect_tx(bar, bytes);
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(0), "r"(0), "r"(r0), "r"(0), "r"(bh), "r"(smem_u32(bar))
        : "memory");
}

// Warps 0-7: softmax (thread tid owns row tid mod 128 of slot tid / 128,
// tensor-memory columns [256 slot, + 256): S in 0-63, P buffers from 64 and 96,
// O from 128); 8-11: dequantizing; 12, 13: S = Q K^T of a slot; 14: O += P V; 15:
// record copies.  They
// meet on mbarriers only (bounded waits): Q written; a K^ / V^ tile written
// (four warps, or a TMA copy and three) and read (MMA commits); S done and P
// written and P V done, per slot and buffer; records landed and read.
template <int D>
__global__ void __launch_bounds__(kCkThreads, 1)
    chunk_attn_kernel(KiviGeom g, KiviDev dv, const __half *__restrict__ Q, const __half *__restrict__ Kn,
                      const __half *__restrict__ Vn, __half *__restrict__ O, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int QB = kCkRows * D * 2, TB = kCkKeys * D * 2, KS = kCkStages;
    constexpr unsigned QLBO = kCkRows * 16, KLBO = kCkKeys * 16, VLBO = D * 16;
    unsigned char *sQ = smem, *sK = sQ + 2 * QB, *sV = sK + KS * TB, *sO = sV + KS * TB, *sR = sO + kCkOut;
    // counts 4 (a slot's or the dequantizing warps): Q [slot], P [slot][buffer],
    // scores read [slot], a meeting, K and V tiles written, records read; 2
    // (both slots' MMAs): K tiles read; 1: the others
    constexpr int N4 = 9 + 2 * KS + kCkMaxRaw, N2 = N4 + KS, NB = N2 + 9 + KS + kCkMaxRaw;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bQ = bars, *const bP = bars + 2, *const bL = bars + 6, *const bX = bars + 8, *const bK = bars + 9,
                    *const bV = bK + KS, *const eR = bV + KS, *const eK = bars + N4, *const bS = bars + N2,
                    *const bF = bS + 2, *const bE = bF + 4, *const eV = bE + 3, *const bR = eV + KS;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;   // a wait ran out: every warp stops
    __shared__ int s_put[2][kCkDq];   // the dequantizing warps' arrivals at K, and V, tiles written
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = a.hg;
    const bool qtma = kCkRows % hg == 0;   // Q's row tiles are boxes of its array
    if (tid < NB) {
        mbar_init(&bars[tid], tid < N4 && !(qtma && tid < 2) ? 4 : tid >= N4 && tid < N2 ? 2 : 1);
        fence_mbar_init();
    }
    if (tid == 0) s_abort = 0;
    if (warp == 0) tc_alloc(&s_taddr, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = s_taddr;
    const volatile int *abort = &s_abort;
    bool ok = true;
    CkWalk walk;
    walk.start(a, blockIdx.x);
    CkSeg sg = {};
    // the segment's first tiles have a record: how many
    auto raw_tiles = [&](int Tq) {
        return max(0, min(sg.x0 + sg.nx, sg.bl.virt((Tq + kCkKeys - 1) / kCkKeys)) - sg.x0);
    };

    if (warp == 8 + kCkDq || warp == 8 + kCkDq + 1) {
        // ---- S = Q K^T of slot e ----
        const int e = __shfl_sync(kFull, warp - (8 + kCkDq), 0);   // (warp-uniform)
        int cnt = 0;            // S of the slot
        CkRing t;
        constexpr uint32_t ID_S = tc_idesc_f16(kCkRows, kCkKeys, 0);
        unsigned qph = 0;
        bool qin = false;       // a copy of Q may be in flight
        const uint64_t dq = tc_desc(sQ + e * QB, QLBO, 128), dk = tc_desc(sK, KLBO, 128);
        while (ok && walk.next(g, a, sg)) {
            const int nx = __reduce_max_sync(kFull, sg.nx);
            const bool mine = sg.nrows - sg.row0 > e * kCkRows;   // (a slot without rows only releases the tiles)
            if (qtma && mine) {   // this segment's Q, once the last one's S is done
                ok = __all_sync(kFull, cnt == 0 || mbar_wait_ab(&bS[e], (unsigned)(cnt - 1) & 1u, abort));
                if (ok && lane == 0)
                    tma_rows(sQ + e * QB, &tmQ, chunk_div(a, sg.row0 + e * kCkRows), sg.i * g.h + sg.j, &bQ[e], QB);
                qin = ok;
            }
            for (int x = 0; x < nx && ok; ++x, t.next(KS)) {
                // its Q and K written, its last scores read
                ok = mbar_wait_ab(&bK[t.s], t.p, abort);
                if (mine)
                    ok = ok && (x > 0 || mbar_wait_ab(&bQ[e], qph, abort)) &&
                         (cnt == 0 || mbar_wait_ab(&bL[e], (unsigned)(cnt - 1) & 1u, abort));
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                if (!mine) {
                    if (lane == 0) mbar_arrive(&eK[t.s]);
                    continue;
                }
                if (x == 0) {
                    qph ^= 1u;
                    qin = false;
                }
                ++cnt;
                tc_fence_after();
                const uint64_t d = dk + (uint32_t)(t.s * (TB >> 4));
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    tc_mma_f16_w(taddr + 256 * e, dq + ((2 * c * QLBO) >> 4), d + ((2 * c * KLBO) >> 4), ID_S, c > 0);
                tc_commit_w(&bS[e]);
                tc_commit_w(&eK[t.s]);
            }
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        // every MMA, commit and copy of this warp has landed before shared
        // memory is given up (bounded)
        if (qin) mbar_wait(&bQ[e], qph);
        tc_commit_w(&bE[e]);
        mbar_wait(&bE[e], 0u);
        __syncwarp();
    } else if (warp == 8 + kCkDq + 2) {
        // ---- O += P V ----
        constexpr uint32_t ID_R = tc_idesc_f16(kCkRows, D, 1), ID_T = tc_idesc_f16(kCkRows, D, 0);
        CkRing tv;
        int cp[2] = {0, 0};     // P V of each slot
        const uint64_t dt = tc_desc(sV, VLBO, 128), dr = tc_desc(sV, 128, KLBO);   // transposed, as rows
        while (ok && walk.next(g, a, sg)) {
            const int nx = __reduce_max_sync(kFull, sg.nx);
            const int slots = __reduce_max_sync(kFull, sg.nrows - sg.row0 > kCkRows ? 2 : 1);
            // tiles with quantized values hold V transposed: the first ones
            const int nt = __reduce_max_sync(kFull, sg.bl.virt((a.Tqv[sg.i] + kCkKeys - 1) / kCkKeys) - sg.x0);
            for (int x = 0; x < nx && ok; ++x) {
                const uint64_t st = (uint32_t)(tv.s * (TB >> 4));
                const uint64_t d = (x < nt ? dt : dr) + st, step = x < nt ? (2 * VLBO) >> 4 : 256 >> 4;
                const uint32_t id = x < nt ? ID_T : ID_R;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (e >= slots || !ok) continue;
                    const int b = cp[e] & 1;
                    ok = mbar_wait_ab(&bP[2 * e + b], (unsigned)(cp[e] >> 1) & 1u, abort) &&
                         (e > 0 || mbar_wait_ab(&bV[tv.s], tv.p, abort));
                    ok = __all_sync(kFull, ok);
                    if (!ok) continue;
                    ++cp[e];
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kCkKeys / 16; ++c)
                        tc_mma_f16_ta_w(taddr + 256 * e + 128, taddr + 256 * e + 64 + 32 * b + 8 * c, d + c * step, id,
                                        x > 0 || c > 0);
                    tc_commit_w(&bF[2 * e + b]);
                    if (e == slots - 1) {
                        tc_commit_w(&eV[tv.s]);
                        tv.next(KS);
                    }
                }
            }
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        tc_commit_w(&bE[2]);
        mbar_wait(&bE[2], 0u);
        __syncwarp();
    } else if (warp == 8 + kCkDq + 3) {
        // ---- records (lane 0 issues) ----
        CkRing r;
        int issued = 0;
        while (walk.next(g, a, sg)) {
            if (lane == 0) {
                const int n = raw_tiles(max(a.Tqk[sg.i], a.Tqv[sg.i]));
                const unsigned char *recs = dv.blk + rec_off(g, sg.i, sg.j, 0);
                for (int y = 0; y < n; ++y, ++issued, r.next(a.rs)) {
                    ok = issued < a.rs || mbar_wait_ab(&eR[r.s], r.p ^ 1u, abort);
                    if (!ok) break;
                    mbar_expect_tx(&bR[r.s], (unsigned)g.rec_bytes);
                    bulk_g2s(sR + (size_t)r.s * g.rec_bytes, recs + (size_t)sg.bl.phys(sg.x0 + y) * g.rec_bytes,
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
            // every copy has landed before shared memory is given up (bounded)
            for (int y = max(0, issued - a.rs); y < issued; ++y) mbar_wait(&bR[y % a.rs], (unsigned)(y / a.rs) & 1u);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---- K^ and V^ tiles ----
        const int w = warp - 8, dt = tid & (32 * kCkDq - 1);
        constexpr int GT = 32 * kCkDq, CPR = D / 8, RPT = kCkKeys * CPR / GT;   // threads, 16-byte chunks a row, a thread's share
        const int lgG = __ffs(g.G) - 1;
        if (a.quit < INT_MAX && w > 0) ok = false;   // (as if a wait had run out)
        int tiles = 0, kin = 0, meets = 0;   // kin: the current tile's K^ is told of
        CkRing t, r;
        // the dequantizing warps meet (a bounded wait, unlike a named barrier)
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bX);
            return __all_sync(kFull, mbar_wait_ab(bX, (unsigned)meets++ & 1u, abort)) != 0;
        };
        while (ok && walk.next(g, a, sg)) {
            const int T = sg.T, n = sg.n, Tqk = a.Tqk[sg.i], Tqv = a.Tqv[sg.i];
            const __half *kwin = dv.Kf + kf_slice(g, sg.i, sg.j), *vwin = dv.Vf + vf_slice(g, sg.i, sg.j);
            const size_t chunk0 = ((size_t)sg.i * g.h + sg.j) * a.n_stride;   // the chunk's first row in K and V
            const int npk = max(0, min(sg.nx, sg.bl.virt(min(Tqk, Tqv) / kCkKeys) - sg.x0));   // fully quantized tiles
            if (g.kbits == 2)
                ok = g.vbits == 2 ? packed_tiles<D, 2, 2>(npk, tiles, t, r, sK, sV, sR, g, a.rs, w, bK, eK, bV, eV, bR, eR, abort)
                                  : packed_tiles<D, 2, 4>(npk, tiles, t, r, sK, sV, sR, g, a.rs, w, bK, eK, bV, eV, bR, eR, abort);
            else
                ok = g.vbits == 2 ? packed_tiles<D, 4, 2>(npk, tiles, t, r, sK, sV, sR, g, a.rs, w, bK, eK, bV, eV, bR, eR, abort)
                                  : packed_tiles<D, 4, 4>(npk, tiles, t, r, sK, sV, sR, g, a.rs, w, bK, eK, bV, eV, bR, eR, abort);
            // a thread's k-th 16-byte chunk of a tile: a warp takes 16
            // rows, 8 rows x 4 chunks at a time (no bank conflicts)
            auto rk = [&](int k) { return 16 * w + k / (CPR / 4) * 8 + (lane & 7); };
            auto ck = [&](int k) { return k % (CPR / 4) * 4 + (lane >> 3); };
            // fp16 row of token tau, in the window or the chunk (zero past the chunk)
            auto row16 = [&](const __half *win, int ring, const __half *chk, int tau, int c) {
                const __half *src = tau < T ? win + (size_t)(tau % ring) * D : chk + (chunk0 + (tau - T)) * D;
                return tau < T + n ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
            };
            // the others: some or all tokens in the window or the chunk
            for (int x = npk; x < sg.nx && ok; ++x, ++tiles, kin = 0, t.next(KS)) {
                const int tb = sg.key0(x);
                unsigned char *kt = sK + t.s * TB, *vt = sV + t.s * TB;
                const bool tma = tb >= T && tb + kCkKeys <= T + n;   // a whole tile of chunk tokens: TMA copies
                const bool raw = tb < max(Tqk, Tqv), kq = tb < Tqk, kall = tb + kCkKeys <= Tqk, vq = tb < Tqv,
                           vall = tb + kCkKeys <= Tqv;
                ok = (tiles < KS || mbar_wait_ab(&eK[t.s], t.p ^ 1u, abort)) && (!raw || mbar_wait_ab(&bR[r.s], r.p, abort));
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                if (tma) {
                    if (warp == 8 && lane == 0)
                        tma_tile(sK + t.s * TB, &tmK, (int)chunk0 + tb - T, &bK[t.s], TB);
                    else if (lane == 0)
                        mbar_arrive(&bK[t.s]);
                    kin = 1;
                    __syncwarp();
                    ok = __all_sync(kFull, tiles < KS || mbar_wait_ab(&eV[t.s], t.p ^ 1u, abort));
                    if (!ok) break;
                    if (warp == 8 && lane == 0)
                        tma_tile(sV + t.s * TB, &tmV, (int)chunk0 + tb - T, &bV[t.s], TB);
                    else if (lane == 0)
                        mbar_arrive(&bV[t.s]);
                    __syncwarp();
                    continue;
                }
                const unsigned char *rec = sR + (size_t)r.s * g.rec_bytes;
                if (kq) {
                    dequant_keys_cold<D, kCkKeys>(kt, rec, g.kbits, g.off_ksz, lgG, w);
                    if (!kall) {   // its window and chunk tokens over the rest
                        if (!(ok = meet())) break;
                        for (int e = dt; e < (tb + kCkKeys - Tqk) * CPR; e += GT) {
                            const int rr = Tqk - tb + e / CPR, c = e % CPR;
                            *reinterpret_cast<uint4 *>(kt + c * KLBO + rr * 16) = row16(kwin, g.R, Kn, tb + rr, c);
                        }
                    }
                } else {
                    uint4 x4[RPT];
#pragma unroll
                    for (int k = 0; k < RPT; ++k)
                        x4[k] = row16(kwin, g.R, Kn, tb + rk(k), ck(k));
#pragma unroll
                    for (int k = 0; k < RPT; ++k)
                        *reinterpret_cast<uint4 *>(kt + ck(k) * KLBO + rk(k) * 16) = x4[k];
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bK[t.s]);
                kin = 1;
                ok = __all_sync(kFull, tiles < KS || mbar_wait_ab(&eV[t.s], t.p ^ 1u, abort));
                if (!ok) break;
                if (vq) {
                    dequant_values_cold<D>(vt, rec, g.vbits, g.off_vc, g.off_vsz, lgG, w);
                    if (!vall) {
                        if (!(ok = meet())) break;
                        for (int e = dt; e < (tb + kCkKeys - Tqv) * CPR; e += GT) {
                            const int rr = Tqv - tb + e / CPR, c = e % CPR;
                            const uint4 v = row16(vwin, g.R + 1, Vn, tb + rr, c);
                            const uint32_t h[4] = {v.x, v.y, v.z, v.w};
                            unsigned char *dst = vt + (rr >> 3) * VLBO + c * 128 + (rr & 7) * 2;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                *reinterpret_cast<uint16_t *>(dst + k * 16) = (uint16_t)(h[k >> 1] >> (16 * (k & 1)));
                        }
                    }
                } else {
                    uint4 x4[RPT];
#pragma unroll
                    for (int k = 0; k < RPT; ++k)
                        x4[k] = row16(vwin, g.R + 1, Vn, tb + rk(k), ck(k));
#pragma unroll
                    for (int k = 0; k < RPT; ++k)
                        *reinterpret_cast<uint4 *>(vt + ck(k) * KLBO + rk(k) * 16) = x4[k];
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bV[t.s]);
                    if (raw) mbar_arrive(&eR[r.s]);
                }
                if (raw) r.next(a.rs);
            }
        }
        if (lane == 0) {
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            s_put[0][w] = tiles + kin;
            s_put[1][w] = tiles;
        }
        __syncwarp();
    } else {
        // ---- the softmax warps ----
        const int slot = tid / kCkRows, rr = tid % kCkRows;
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = taddr + 256 * slot + lane_off, tO = tS + 128;
        const float sl2 = 1.4426950408889634f / sqrtf((float)D);   // log2(e) / sqrt(d)
        const int W = a.vis.window, sinks = a.vis.sinks;
        int cnt = 0;   // this slot's tiles so far
        while (walk.next(g, a, sg)) {
            const int srow = sg.row0 + slot * kCkRows, row = srow + rr;   // the slot's first row, this thread's
            const bool in = row < sg.nrows;
            if (srow >= sg.nrows) continue;   // no rows in this slot
            if (!qtma) {
                // Q: row (r, e) from head e of token r; rows past the chunk
                // are zero.  (This slot's S MMAs have read the last
                // segment's.)  A warp takes its 32 rows, 8 rows x 4 chunks at
                // a time (no bank conflicts), loads ahead of stores.
                auto qr = [&](int k) { return 32 * (warp & 3) + k / (D / 32) * 8 + (lane & 7); };
                auto qc = [&](int k) { return k % (D / 32) * 4 + (lane >> 3); };
#pragma unroll 1
                for (int k0 = 0; k0 < D / 8; k0 += 8) {
                    uint4 v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int rw = min(srow + qr(k0 + k), sg.nrows - 1), tok = chunk_div(a, rw);
                        v[k] = *reinterpret_cast<const uint4 *>(
                            Q + (((size_t)sg.i * a.hq + sg.j * hg + rw - tok * hg) * a.n_stride + tok) * D + 8 * qc(k0 + k));
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (srow + qr(k0 + k) >= sg.nrows) v[k] = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(sQ + slot * QB + qc(k0 + k) * QLBO + qr(k0 + k) * 16) = v[k];
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bQ[slot]);
            }
            const int pos = sg.T + chunk_div(a, row), ps0 = sg.T + chunk_div(a, srow),
                      ps1 = sg.T + chunk_div(a, srow + kCkRows - 1);
            // minus the log2 weight of a score of zero (the row's reference less
            // the lift; -inf: nothing seen yet), and the weights' sum
            float ref = -INFINITY, lsum = 0.f;
            for (int x = 0; x < sg.nx; ++x, ++cnt) {
                const int b = cnt & 1, key0 = sg.key0(x);
                ok = __all_sync(kFull, mbar_wait_ab(&bS[slot], (unsigned)cnt & 1u, abort));
                if (!ok) break;
                tc_fence_after();
                uint32_t r[2][32];   // this row's 64 scores
                tc_ld32(tS, r[0]);
                tc_ld32(tS + 32, r[1]);
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bL[slot]);
                // this P buffer's last P V has read its weights (polled ahead: most often true)
                const bool pf = cnt < 2 || mbar_test(&bF[2 * slot + b], (unsigned)((cnt >> 1) + 1) & 1u);
                if (key0 + kCkKeys - 1 > ps0 || (W > 0 && key0 <= ps1 - W && key0 + kCkKeys > sinks)) {
                    // some row of the slot does not see the whole tile
                    const uint32_t h0 = ck_hidden32(key0, pos, W, sinks), h1 = ck_hidden32(key0 + 32, pos, W, sinks);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if ((h0 >> c) & 1u) r[0][c] = 0xff800000u;
                        if ((h1 >> c) & 1u) r[1][c] = 0xff800000u;
                    }
                }
                float m8[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) m8[c] = __uint_as_float(r[0][c]);
#pragma unroll
                for (int c = 8; c < 64; ++c) m8[c & 7] = fmaxf(m8[c & 7], __uint_as_float(r[c >> 5][c & 31]));
                const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                       fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                // lazy rescale: only when the maximum grew by more than 2^8 in weight
                const bool grow = mx != -INFINITY && (ref == -INFINITY || fmaf(mx, sl2, -ref) > kCkLift + kCkLag);
                const float up = fmaf(mx, sl2, -kCkLift);
                const float alpha = grow && ref != -INFINITY ? ex2(ref - up) : 1.f;
                if (grow) ref = up;
                const float ms = ref == -INFINITY ? 0.f : ref;   // (nothing seen yet: weights 0)
                const unsigned long long sc2 = ck_f2(sl2, sl2), ms2 = ck_f2(-ms, -ms);
                unsigned long long l2[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t pw[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float y0, y1;
                    ck_f2(ck_fma2(ck_f2(__uint_as_float(r[c >> 4][2 * c & 31]), __uint_as_float(r[c >> 4][(2 * c & 31) + 1])),
                                  sc2, ms2), y0, y1);
                    y0 = ex2(y0);
                    y1 = ex2(y1);
                    l2[c & 3] = ck_add2(l2[c & 3], ck_f2(y0, y1));
                    pw[c] = ck_pack(y0, y1);
                }
                float l0, l1;
                ck_f2(ck_add2(ck_add2(l2[0], l2[1]), ck_add2(l2[2], l2[3])), l0, l1);
                lsum = lsum * alpha + (l0 + l1);
                if (x > 0 && __any_sync(kFull, alpha != 1.f)) {   // rescale O, once P V of tile x - 1 is in
                    ok = __all_sync(kFull, mbar_wait_ab(&bF[2 * slot + (b ^ 1)], (unsigned)((cnt - 1) >> 1) & 1u, abort));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc_ld32(tO + c0, o);
                        tc_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                        tc_st32(tO + c0, o);
                    }
                }
                ok = __all_sync(kFull, pf || mbar_wait_ab(&bF[2 * slot + b], (unsigned)((cnt >> 1) + 1) & 1u, abort));
                if (!ok) break;
                tc_fence_after();
                tc_st32(tS + 64 + 32 * b, pw);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bP[2 * slot + b]);
            }
            // the last two P V
            for (int y = max(cnt - 2, cnt - sg.nx); y < cnt && ok; ++y)
                ok = __all_sync(kFull, mbar_wait_ab(&bF[2 * slot + (y & 1)], (unsigned)(y >> 1) & 1u, abort));
            if (!ok) break;
            tc_fence_after();
            if (sg.nx < sg.nt) {   // this CTA's partial of the row
                const size_t pr = (size_t)(2 * blockIdx.x + (sg.x0 == 0 ? 1 : 0)) * kCkTileRows + slot * kCkRows + rr;
                if (in) reinterpret_cast<float2 *>(a.ml)[pr] = make_float2(ref, lsum);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tc_ld32(tO + c0, o);
                    tc_wait_ld();
                    if (in)
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            *reinterpret_cast<uint4 *>(a.acc + pr * D + c0 + c) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                }
            } else {
                // 32 columns at a time through shared memory (16-byte chunk c of
                // row r at chunk c ^ (r / 2 mod 4) of it: no bank conflicts),
                // so that a store covers 64 consecutive bytes of 8 rows
                const float r = 1.f / lsum;
                unsigned char *st = sO + warp * (32 * 64);
                const int q8 = lane >> 2, c4 = lane & 3, row32 = srow + 32 * (warp & 3);
                size_t orow[4];   // the rows this lane stores
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int rw = min(row32 + 8 * k + q8, sg.nrows - 1), tok = chunk_div(a, rw);
                    orow[k] = (((size_t)sg.i * a.hq + sg.j * hg + rw - tok * hg) * a.n_stride + tok) * D + 8 * c4;
                }
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tc_ld32(tO + c0, o);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4 *>(st + lane * 64 + ((c ^ (lane >> 1)) & 3) * 16) =
                            make_uint4(ck_pack(__uint_as_float(o[8 * c]) * r, __uint_as_float(o[8 * c + 1]) * r),
                                       ck_pack(__uint_as_float(o[8 * c + 2]) * r, __uint_as_float(o[8 * c + 3]) * r),
                                       ck_pack(__uint_as_float(o[8 * c + 4]) * r, __uint_as_float(o[8 * c + 5]) * r),
                                       ck_pack(__uint_as_float(o[8 * c + 6]) * r, __uint_as_float(o[8 * c + 7]) * r));
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int q = 8 * k + q8;
                        const uint4 v = *reinterpret_cast<const uint4 *>(st + q * 64 + ((c4 ^ (q >> 1)) & 3) * 16);
                        if (row32 + q < sg.nrows) *reinterpret_cast<uint4 *>(O + orow[k] + c0) = v;
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (s_abort && tid == 32 * 8) drain_tiles<KS>(s_put, bK, bV);
    if (warp == 0) tc_dealloc(taddr, 512);
}

}  // namespace
