// kivi_chunk_attn_impl.cuh -- attention of a chunk of new tokens over the
// quantized cache and the chunk itself, on the 5th-generation tensor cores.
//
// Mathematics.  Row (r, e) of kv head j is query head j hg + e of chunk token
// r, at position p = T + r:
//   out = sum_s softmax_s(q . K^_s / sqrt(d)) V^_s   over the visible s <= p,
// K^_s = scale code + zero for the quantized tokens ("Literature audit --
// Group 2", section 1 KIVI, core algorithm item 5), the fp16 rows for the
// window's and the chunk's.  All hg heads of a kv head share its tokens, so
// the rows (r, e) are one list, row index r hg + e, cut into CTA tiles of
// 128 NH rows; a one-token chunk is a tile of hg rows.
//
// Per 64-token tile the CTA restores K^ and V^ once as fp16 tiles in shared
// memory (dequantizing warps), S = Q K^T and O += P V run on tcgen05 with
// S, P and O in tensor memory and one thread a row doing the online softmax,
// as in the prompt's attention.  K^ and V^ round once to fp16 (2^-11
// relative a value, as the weights P do): the two-term operands that the
// one-token decode uses would double the MMAs, and the errors of the rounded
// values are independent, so they average like the values themselves.
//
// A tile's record (packed codes, scales, zeros) comes into a ring of
// shared-memory stages with one bulk copy, several tiles ahead.  The four
// dequantizing warps write K^ as rows of tokens and V^ as rows of channels
// (V^ transposed: the value words hold two tokens of one channel, so each
// half2 they yield is contiguous along tokens); both stores are free of bank
// conflicts, and the MMA's descriptor takes V^ K-major.  Tiles of fp16
// tokens are copied as rows, and the MMA takes V MN-major.
//
// Long caches with few rows: each row tile's tokens are split into pieces, a
// CTA each, which leave unnormalized partials (max, sum, O) that a second
// kernel joins.
#pragma once
#include <cuda_fp16.h>

#include "kivi_async.cuh"
#include "kivi_chunk.cuh"
#include "kivi_internal.cuh"
#include "kivi_mma.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_unpack.cuh"

namespace {

constexpr int kCkRows = 128, kCkKeys = KIVI_KBLK;
constexpr int kCkStages = 3;     // K^ / V^ tiles in flight
constexpr int kCkMaxRaw = 8;     // records in flight
constexpr int kCkDq = 4;         // dequantizing warps

__device__ __forceinline__ uint32_t ck_pack(float lo, float hi) {
    return h2u(__floats2half2_rn(lo, hi));
}
// s code + z of two values, the code from off + code (exact)
__device__ __forceinline__ uint32_t ck_affine(uint32_t x, float off, uint32_t s, uint32_t z) {
    return h2u(__hfma2(__hsub2(u2h(x), __float2half2_rn(off)), u2h(s), u2h(z)));
}

// K^ of a record's 64 tokens: chunk-major tile [64 tokens][D], 16-byte chunk
// c of token r at byte c 1024 + r 16.  Warp w of the kCkDq takes the
// 16-channel steps w, w + kCkDq, ...; a lane's half2 (two channels of one token) are
// the lanes t = 0..3 of one 16-byte chunk: 128 consecutive bytes a store.
template <int D, int KB>
__device__ __forceinline__ void dequant_keys(unsigned char *tile, const unsigned char *rec, int off_ksz, int lgG,
                                             int w) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const __half *ksz = reinterpret_cast<const __half *>(rec + off_ksz) + tq * (D / 4);
    unsigned char *dst = tile + gq * 16 + tq * 4;
    constexpr int NW = KB / 2;   // words of a channel pair
    // one 16-channel step a turn, not unrolled (see dequant_values)
#pragma unroll 1
    for (int j = w; j < D / 16; j += kCkDq) {
        // every load before the first store: the compiler keeps their order
        uint32_t W[2 * NW];
        const unsigned char *pw = rec + (size_t)((j * 2 * NW) >> 2) * 512 + lane * 16 + ((j * 2 * NW) & 3) * 4;
        if (KB == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(pw);
            W[0] = v.x;
            W[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(pw);
            W[0] = v.x;
            W[1] = v.y;
            W[NW] = v.z;
            W[2 * NW - 1] = v.w;
        }
        uint2 sv[4], zv[4];
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {   // 16 tokens share a group row
            const __half *row = ksz + (((16 * qd) >> lgG) * 2) * D + 4 * j;
            sv[qd] = *reinterpret_cast<const uint2 *>(row);
            zv[qd] = *reinterpret_cast<const uint2 *>(row + D);
        }
        unsigned char *p = dst + (size_t)(2 * j) * (kCkKeys * 16);
#pragma unroll
        for (int pos = 0; pos < 8; ++pos) {
            const int wi = KB == 2 ? 0 : pos >> 2, r = KB == 2 ? pos : pos & 3;
            const float off = slot_offset<KB, true>(r);
            const uint2 sc = sv[pos >> 1], z = zv[pos >> 1];
            *reinterpret_cast<uint32_t *>(p + pos * 128) = ck_affine(unpack<KB, true>(W[wi], r), off, sc.x, z.x);
            *reinterpret_cast<uint32_t *>(p + kCkKeys * 16 + pos * 128) =
                ck_affine(unpack<KB, true>(W[NW + wi], r), off, sc.y, z.y);
        }
    }
}

// V^ of a record's 64 tokens, transposed: chunk-major tile [D channels][64
// tokens], tokens 8 k .. 8 k + 7 of channel c at byte k D 16 + c 16.  Warp w
// takes value block w (16 tokens).
template <int D, int VB>
__device__ __forceinline__ void dequant_values(unsigned char *tile, const unsigned char *rec, int off_vc, int off_vsz,
                                               int lgG, int w) {
    constexpr int WL = D * VB / 64, CS = WL < 4 ? WL : 4, NWV = D * VB / 128, CPH = 16 / VB;
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int ngi = D >> lgG;
    const uint32_t *words = reinterpret_cast<const uint32_t *>(rec + off_vc) + (size_t)w * (D * VB / 2) + lane * CS;
    const __half *vsz = reinterpret_cast<const __half *>(rec + off_vsz) + (size_t)w * (2 * ngi * 16) + 4 * tq;
    unsigned char *dst = tile + (size_t)(2 * w) * (D * 16) + gq * 16 + tq * 4;
    // one word (CPH channel steps of 8) a turn, not unrolled: short code
    // stays in the instruction cache beside the softmax warps'
#pragma unroll 1
    for (int wi = 0; wi < NWV; ++wi, dst += CPH * 128) {
        // every load before the first store: the compiler keeps their order
        const int u1 = NWV + wi;   // tokens 2 t, 2 t + 1: word wi; + 8: word u1
        const uint32_t W0 = words[wi / CS * 32 * CS + wi % CS], W1 = words[u1 / CS * 32 * CS + u1 % CS];
        uint2 sv[CPH / 2], zv[CPH / 2];
#pragma unroll
        for (int q = 0; q < CPH / 2; ++q) {   // 16 channels share a group row
            const int gi = (16 * (wi * (CPH / 2) + q)) >> lgG;
            sv[q] = *reinterpret_cast<const uint2 *>(vsz + gi * 16);
            zv[q] = *reinterpret_cast<const uint2 *>(vsz + (ngi + gi) * 16);
        }
#pragma unroll
        for (int r = 0; r < CPH; ++r) {
            const float off = slot_offset<VB, false>(r);
            *reinterpret_cast<uint32_t *>(dst + r * 128) =
                ck_affine(unpack<VB, false>(W0, r), off, sv[r >> 1].x, zv[r >> 1].x);
            *reinterpret_cast<uint32_t *>(dst + D * 16 + r * 128) =
                ck_affine(unpack<VB, false>(W1, r), off, sv[r >> 1].y, zv[r >> 1].y);
        }
    }
}

// position in a ring of stages, and the phase its next use completes
struct CkRing {
    int s = 0;
    unsigned p = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            p ^= 1u;
        }
    }
};

// One dequantizing warp's share of the tiles [0, n) of a piece, all of them
// fully quantized: the loop that most of a long cache runs in, kept apart
// (and short) from the tiles with fp16 tokens.  False if a wait ran out.
template <int D, int KB, int VB>
__device__ __forceinline__ bool packed_tiles(int n, CkRing &t, CkRing &r, unsigned char *sK, unsigned char *sV,
                                             const unsigned char *sR, const KiviGeom &g, int rs, int w, uint64_t *bT,
                                             uint64_t *eT, uint64_t *bR, uint64_t *eR, const volatile int *abort) {
    constexpr int TB = kCkKeys * D * 2;
    const int lane = threadIdx.x & 31, lgG = __ffs(g.G) - 1;
    for (int x = 0; x < n; ++x) {
        const bool ok = (x < kCkStages || mbar_wait_ab(&eT[t.s], t.p ^ 1u, abort)) && mbar_wait_ab(&bR[r.s], r.p, abort);
        if (!__all_sync(0xffffffffu, ok)) return false;
        const unsigned char *rec = sR + (size_t)r.s * g.rec_bytes;
        dequant_keys<D, KB>(sK + t.s * TB, rec, g.off_ksz, lgG, w);
        dequant_values<D, VB>(sV + t.s * TB, rec, g.off_vc, g.off_vsz, lgG, w);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bT[t.s]);
            mbar_arrive(&eR[r.s]);
        }
        t.next(kCkStages);
        r.next(rs);
    }
    return true;
}

// Warps: 4 NH of softmax (thread tid owns row tid mod 128 of slot tid / 128,
// tensor-memory columns [256 slot, + 256): S / P buffers in 0-63 and 64-127,
// O from 128), kCkDq dequantizing, one issuing S = Q K^T, one O += P V, one
// copying records (an issue and its wait take long enough to hold a
// dequantizing warp back).
// They meet on mbarriers (bounded waits): a tile's K^ / V^ written,
// read (MMA commits), S done, P written, P V done; records landed and read.
template <int D, int NH>
__global__ void __launch_bounds__(32 * (4 * NH + kCkDq + 3), 1)
    chunk_attn_kernel(KiviGeom g, KiviDev dv, const __half *__restrict__ Q, const __half *__restrict__ Kn,
                      const __half *__restrict__ Vn, __half *__restrict__ O, const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int QB = kCkRows * D * 2, TB = kCkKeys * D * 2;
    constexpr unsigned QLBO = kCkRows * 16, KLBO = kCkKeys * 16, VLBO = D * 16;
    constexpr int NSW = 4 * NH, CR = NH * kCkRows, TS = kCkStages;
    unsigned char *sQ = smem, *sK = sQ + NH * QB, *sV = sK + TS * TB, *sR = sV + TS * TB;
    constexpr int NB = 7 + 2 * TS + 2 * kCkMaxRaw;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bS = bars, *const bF = bars + 2, *const bP = bars + 4, *const bT = bars + 6, *const eT = bT + TS,
                    *const bR = eT + TS, *const eR = bR + kCkMaxRaw, *const bX = eR + kCkMaxRaw;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;   // a wait ran out: every warp stops
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = a.hq / g.h;

    // the CTA's (sequence, kv head, row tile, piece)
    int i = 0;
    for (int lo = 0, hi = g.b; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (a.start[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
        i = lo;
    }
    const int T = a.T[i], Tqk = a.Tqk[i], Tqv = a.Tqv[i], n = a.n[i];
    const int nrows = n * hg, mt = (nrows + CR - 1) / CR;
    const int sp = (a.start[i + 1] - a.start[i]) / (g.h * mt);
    int rem = blockIdx.x - a.start[i];
    const int j = rem / (mt * sp);
    rem -= j * mt * sp;
    const int row0 = rem / sp * CR, piece = rem % sp;
    const int p0 = T + row0 / hg, p1 = T + min(n - 1, (row0 + CR - 1) / hg);   // first and last position
    const BlockList bl = visible_blocks(a.vis, p0);
    const int nt = bl.virt(p1 / kCkKeys + 1);
    const int x0 = (int)((long long)nt * piece / sp), nx = (int)((long long)nt * (piece + 1) / sp) - x0;   // its tiles
    auto tile0 = [&](int x) { return bl.phys(x0 + x) * kCkKeys; };   // first token of tile x

    if (nx == 0) {   // an empty piece (fewer tiles than pieces)
        for (int r = tid; r < CR; r += blockDim.x)
            reinterpret_cast<float2 *>(a.ml)[(size_t)blockIdx.x * CR + r] = make_float2(-INFINITY, 0.f);
        return;
    }
    if (tid == 0) {
        for (int k = 0; k < NB; ++k) {
            const bool written = k >= 6 && k < 6 + TS, read_raw = k >= 6 + 2 * TS + kCkMaxRaw;
            mbar_init(&bars[k], k == 4 || k == 5 ? NSW : written || read_raw ? kCkDq : 1);
        }
        fence_mbar_init();
        s_abort = 0;
    }
    __syncthreads();
    if (warp == 0) tc_alloc(&s_taddr, 256 * NH);
    // Q: row (r, e) from head e of token r; rows past the chunk are zero
    for (int e = tid; e < CR * (D / 8); e += blockDim.x) {
        const int rr = e / (D / 8), c = e % (D / 8), row = row0 + rr;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < nrows)
            v = *reinterpret_cast<const uint4 *>(
                Q + (((size_t)i * a.hq + j * hg + row % hg) * a.n_stride + row / hg) * D + 8 * c);
        *reinterpret_cast<uint4 *>(sQ + (rr / kCkRows) * QB + c * QLBO + (rr % kCkRows) * 16) = v;
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = s_taddr;
    const volatile int *abort = &s_abort;
    bool ok = true;
    const int nraw = min(nx, max(0, bl.virt((max(Tqk, Tqv) + kCkKeys - 1) / kCkKeys) - x0));   // tiles with records
    if (warp == NSW + kCkDq + 2) {
        // ---- records (lane 0) ----
        if (lane == 0) {
            const unsigned char *recs = dv.blk + rec_off(g, i, j, 0);
            CkRing r;
            int x = 0;
            for (; x < nraw; ++x, r.next(a.rs)) {
                ok = x < a.rs || mbar_wait_ab(&eR[r.s], r.p ^ 1u, abort);   // read
                if (!ok) break;
                mbar_expect_tx(&bR[r.s], (unsigned)g.rec_bytes);
                bulk_g2s(sR + (size_t)r.s * g.rec_bytes, recs + (size_t)(tile0(x) / kCkKeys) * g.rec_bytes,
                         (unsigned)g.rec_bytes, &bR[r.s]);
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            // every copy has landed before shared memory is given up (bounded)
            for (int y = max(0, x - a.rs); y < x; ++y) mbar_wait(&bR[y % a.rs], (unsigned)(y / a.rs) & 1u);
        }
        __syncwarp();
    } else if (warp == NSW + kCkDq) {
        // ---- S = Q K^T (lane 0) ----
        if (lane == 0) {
            constexpr uint32_t ID_S = tc_idesc_f16(kCkRows, kCkKeys, 0);
            CkRing t;
            int x = 0;
            for (; x < nx; ++x, t.next(TS)) {
                // its tile written, its S buffer free (P V of tile x - 2 read its weights there)
                ok = mbar_wait_ab(&bT[t.s], t.p, abort) &&
                     (x < 2 || mbar_wait_ab(&bF[x & 1], (unsigned)((x >> 1) + 1) & 1u, abort));
                if (!ok) break;
                tc_fence_after();
                const unsigned char *k = sK + t.s * TB;
#pragma unroll
                for (int e = 0; e < NH; ++e)
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)
                        tc_mma_f16(taddr + 256 * e + 64 * (x & 1), tc_desc(sQ + e * QB + 2 * c * QLBO, QLBO, 128),
                                   tc_desc(k + 2 * c * KLBO, KLBO, 128), ID_S, c > 0);
                tc_commit(&bS[x & 1]);
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            // every commit has landed before shared memory is given up (bounded)
            for (int y = max(0, x - 2); y < x; ++y) mbar_wait(&bS[y & 1], (unsigned)(y >> 1) & 1u);
        }
        __syncwarp();
    } else if (warp == NSW + kCkDq + 1) {
        // ---- O += P V (lane 0) ----
        if (lane == 0) {
            constexpr uint32_t ID_R = tc_idesc_f16(kCkRows, D, 1), ID_T = tc_idesc_f16(kCkRows, D, 0);
            CkRing t;
            int x = 0;
            for (; x < nx; ++x, t.next(TS)) {
                const bool transposed = tile0(x) < Tqv;
                // (its P written: S read the tile, which was written before)
                ok = mbar_wait_ab(&bP[x & 1], (unsigned)(x >> 1) & 1u, abort) && mbar_wait_ab(&bT[t.s], t.p, abort);
                if (!ok) break;
                tc_fence_after();
                const unsigned char *v = sV + t.s * TB;
#pragma unroll
                for (int e = 0; e < NH; ++e)
#pragma unroll
                    for (int c = 0; c < kCkKeys / 16; ++c)
                        tc_mma_f16_ta(taddr + 256 * e + 128, taddr + 256 * e + 64 * (x & 1) + 8 * c,
                                      transposed ? tc_desc(v + 2 * c * VLBO, VLBO, 128)
                                                 : tc_desc(v + 256 * c, 128, KLBO),
                                      transposed ? ID_T : ID_R, x > 0 || c > 0);
                tc_commit(&bF[x & 1]);
                tc_commit(&eT[t.s]);
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            for (int y = max(0, x - 2); y < x; ++y) mbar_wait(&bF[y & 1], (unsigned)(y >> 1) & 1u);
            for (int y = max(0, x - TS); y < x; ++y) mbar_wait(&eT[y % TS], (unsigned)(y / TS) & 1u);
        }
        __syncwarp();
    } else if (warp >= NSW) {
        // ---- K^ and V^ tiles ----
        const int w = warp - NSW, dt = tid - 32 * NSW;   // dt: 0 .. 127
        const int lgG = __ffs(g.G) - 1;
        const __half *kwin = dv.Kf + kf_slice(g, i, j), *vwin = dv.Vf + vf_slice(g, i, j);
        const __half *kch = Kn + ((size_t)i * g.h + j) * a.n_stride * D, *vch = Vn + ((size_t)i * g.h + j) * a.n_stride * D;
        // the dequantizing warps meet (a bounded wait, unlike a named barrier)
        int meets = 0;
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bX);
            return __all_sync(0xffffffffu, mbar_wait_ab(bX, (unsigned)meets++ & 1u, abort)) != 0;
        };
        // fp16 rows: token tau's row in the window or the chunk (zero past the chunk)
        auto row16 = [&](const __half *win, int ring, const __half *chk, int tau, int c) {
            const __half *src = tau < T ? win + (size_t)(tau % ring) * D : chk + (size_t)(tau - T) * D;
            return tau < T + n ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        };
        constexpr int CPR = D / 8, RPT = kCkKeys * CPR / 128;   // 16-byte chunks a row; a thread's share of a tile
        CkRing t, r;   // this tile's and record's stages
        const int npk = min(nx, max(0, bl.virt(min(Tqk, Tqv) / kCkKeys) - x0));   // fully quantized tiles
        if (g.kbits == 2)
            ok = g.vbits == 2 ? packed_tiles<D, 2, 2>(npk, t, r, sK, sV, sR, g, a.rs, w, bT, eT, bR, eR, abort)
                              : packed_tiles<D, 2, 4>(npk, t, r, sK, sV, sR, g, a.rs, w, bT, eT, bR, eR, abort);
        else
            ok = g.vbits == 2 ? packed_tiles<D, 4, 2>(npk, t, r, sK, sV, sR, g, a.rs, w, bT, eT, bR, eR, abort)
                              : packed_tiles<D, 4, 4>(npk, t, r, sK, sV, sR, g, a.rs, w, bT, eT, bR, eR, abort);
        // the others: some or all tokens in the window or the chunk
        for (int x = npk; x < nx && ok; ++x, t.next(TS)) {
            const int tb = tile0(x);
            unsigned char *kt = sK + t.s * TB, *vt = sV + t.s * TB;
            const bool raw = x < nraw;
            const bool kq = tb < Tqk, kall = tb + kCkKeys <= Tqk, vq = tb < Tqv, vall = tb + kCkKeys <= Tqv;
            uint4 kr[RPT], vr[RPT];   // fp16 tiles: loads in flight before the waits
            if (!kq)
#pragma unroll
                for (int k = 0; k < RPT; ++k)
                    kr[k] = row16(kwin, g.R, kch, tb + (dt + 128 * k) / CPR, (dt + 128 * k) % CPR);
            if (!vq)
#pragma unroll
                for (int k = 0; k < RPT; ++k)
                    vr[k] = row16(vwin, g.R + 1, vch, tb + (dt + 128 * k) / CPR, (dt + 128 * k) % CPR);
            ok = (x < TS || mbar_wait_ab(&eT[t.s], t.p ^ 1u, abort)) && (!raw || mbar_wait_ab(&bR[r.s], r.p, abort));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const unsigned char *rec = sR + (size_t)r.s * g.rec_bytes;
            if (kq) {
                if (g.kbits == 2) dequant_keys<D, 2>(kt, rec, g.off_ksz, lgG, w);
                else dequant_keys<D, 4>(kt, rec, g.off_ksz, lgG, w);
                if (!kall) {   // its window and chunk tokens over the rest
                    if (!(ok = meet())) break;
                    for (int e = dt; e < (tb + kCkKeys - Tqk) * CPR; e += 128) {
                        const int r = Tqk - tb + e / CPR, c = e % CPR;
                        *reinterpret_cast<uint4 *>(kt + c * KLBO + r * 16) = row16(kwin, g.R, kch, tb + r, c);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < RPT; ++k)
                    *reinterpret_cast<uint4 *>(kt + ((dt + 128 * k) % CPR) * KLBO + (dt + 128 * k) / CPR * 16) = kr[k];
            }
            if (vq) {
                if (g.vbits == 2) dequant_values<D, 2>(vt, rec, g.off_vc, g.off_vsz, lgG, w);
                else dequant_values<D, 4>(vt, rec, g.off_vc, g.off_vsz, lgG, w);
                if (!vall) {
                    if (!(ok = meet())) break;
                    for (int e = dt; e < (tb + kCkKeys - Tqv) * CPR; e += 128) {
                        const int r = Tqv - tb + e / CPR, c = e % CPR;
                        const uint4 v = row16(vwin, g.R + 1, vch, tb + r, c);
                        const uint32_t h[4] = {v.x, v.y, v.z, v.w};
                        unsigned char *dst = vt + (r >> 3) * VLBO + c * 128 + (r & 7) * 2;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<uint16_t *>(dst + k * 16) = (uint16_t)(h[k >> 1] >> (16 * (k & 1)));
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < RPT; ++k)
                    *reinterpret_cast<uint4 *>(vt + ((dt + 128 * k) % CPR) * KLBO + (dt + 128 * k) / CPR * 16) = vr[k];
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bT[t.s]);
                if (raw) mbar_arrive(&eR[r.s]);
            }
            if (raw) r.next(a.rs);
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        __syncwarp();
    } else {
        // ---- the softmax warps ----
        const int slot = tid / kCkRows, rr = tid % kCkRows;
        const uint32_t tH = taddr + 256 * slot, tO = tH + 128;
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const float sl2 = 1.4426950408889634f / sqrtf((float)D);   // log2(e) / sqrt(d)
        const int row = row0 + slot * kCkRows + rr, pos = T + row / hg;
        const int ps0 = T + (row0 + slot * kCkRows) / hg, ps1 = T + (row0 + slot * kCkRows + kCkRows - 1) / hg;
        const int W = a.vis.window, sinks = a.vis.sinks;
        float mref = -INFINITY, lsum = 0.f;   // the row's reference maximum (raw score units) and weight sum
        for (int x = 0; x < nx; ++x) {
            const int b = x & 1, key0 = tile0(x);
            ok = __all_sync(0xffffffffu, mbar_wait_ab(&bS[b], (unsigned)(x >> 1) & 1u, abort));
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = tH + 64 * b;
            uint32_t sr[2][32];
            tc_ld32(tS + lane_off, sr[0]);
            tc_ld32(tS + lane_off + 32, sr[1]);
            tc_wait_ld();
            float sc[64];
            if (key0 + kCkKeys - 1 > ps0 || (W > 0 && key0 <= ps1 - W && key0 + kCkKeys > sinks)) {
                const int lo = W > 0 ? pos - W : -1;   // tokens [sinks, lo] are hidden
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    const int key = key0 + c;
                    const bool hid = key > pos || (key <= lo && key >= sinks);
                    sc[c] = hid ? -INFINITY : __uint_as_float(sr[c >> 5][c & 31]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 64; ++c) sc[c] = __uint_as_float(sr[c >> 5][c & 31]);
            }
            float m8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = sc[k];
#pragma unroll
            for (int c = 8; c < 64; ++c) m8[c & 7] = fmaxf(m8[c & 7], sc[c]);
            const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                   fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
            // lazy rescale: only when the maximum grew by more than 2^8 in weight
            const bool grow = mx != -INFINITY && (mref == -INFINITY || (mx - mref) * sl2 > 8.f);
            const float alpha = grow && mref != -INFINITY ? ex2((mref - mx) * sl2) : 1.f;
            if (grow) mref = mx;
            const float ms = mref == -INFINITY ? 0.f : mref * sl2;   // (nothing seen yet: weights 0)
            uint32_t pw[32];
            float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const float e0 = ex2(fmaf(sc[2 * c], sl2, -ms)), e1 = ex2(fmaf(sc[2 * c + 1], sl2, -ms));
                l4[c & 3] += e0 + e1;
                pw[c] = ck_pack(e0, e1);
            }
            lsum = lsum * alpha + ((l4[0] + l4[1]) + (l4[2] + l4[3]));
            if (x > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {   // rescale O, once P V of tile x - 1 is in
                ok = __all_sync(0xffffffffu, mbar_wait_ab(&bF[b ^ 1], (unsigned)((x - 1) >> 1) & 1u, abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tc_ld32(tO + lane_off + c0, o);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                    tc_st32(tO + lane_off + c0, o);
                }
            }
            tc_st32(tS + lane_off, pw);   // P over the first 32 columns of its S buffer
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bP[b]);
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_ab(&bF[(nx - 1) & 1], (unsigned)((nx - 1) >> 1) & 1u, abort));
        if (!ok) {
            if (lane == 0) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
        } else {
            tc_fence_after();
            const bool in = row < nrows;
            if (sp > 1) {   // this piece's partial of the row
                const size_t pr = (size_t)blockIdx.x * CR + slot * kCkRows + rr;
                if (in) reinterpret_cast<float2 *>(a.ml)[pr] = make_float2(mref * sl2, lsum);
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tc_ld32(tO + lane_off + c0, o);
                    tc_wait_ld();
                    if (in)
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            *reinterpret_cast<uint4 *>(a.acc + pr * D + c0 + c) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                }
            } else {
                const float r = 1.f / lsum;
                const int rc = min(row, nrows - 1);
                __half *orow = O + (((size_t)i * a.hq + j * hg + rc % hg) * a.n_stride + rc / hg) * D;
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tc_ld32(tO + lane_off + c0, o);
                    tc_wait_ld();
                    if (in)
#pragma unroll
                        for (int c = 0; c < 32; c += 8)
                            *reinterpret_cast<uint4 *>(orow + c0 + c) =
                                make_uint4(ck_pack(__uint_as_float(o[c]) * r, __uint_as_float(o[c + 1]) * r),
                                           ck_pack(__uint_as_float(o[c + 2]) * r, __uint_as_float(o[c + 3]) * r),
                                           ck_pack(__uint_as_float(o[c + 4]) * r, __uint_as_float(o[c + 5]) * r),
                                           ck_pack(__uint_as_float(o[c + 6]) * r, __uint_as_float(o[c + 7]) * r));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(taddr, 256 * NH);
}

// Joins the pieces of one row a warp: weights 2^(m_k - M), M the largest m.
template <int D>
__global__ void __launch_bounds__(256)
    chunk_join_kernel(KiviGeom g, __half *__restrict__ O, const __grid_constant__ ChunkArgs a, int CR) {
    constexpr int V = D / 32;
    const int i = blockIdx.z, j = blockIdx.y, lane = threadIdx.x & 31;
    const int hg = a.hq / g.h, nrows = a.n[i] * hg, row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= nrows) return;
    const int mt = (nrows + CR - 1) / CR, sp = (a.start[i + 1] - a.start[i]) / (g.h * mt);
    if (sp <= 1) return;
    const size_t pr = ((size_t)a.start[i] + ((size_t)j * mt + row / CR) * sp) * CR + row % CR;   // + k CR
    const float2 *ml = reinterpret_cast<const float2 *>(a.ml);
    float M = -INFINITY;
    for (int k = lane; k < sp; k += 32) M = fmaxf(M, ml[pr + (size_t)k * CR].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
    for (int k = 0; k < sp; ++k) {
        const float2 m = ml[pr + (size_t)k * CR];
        if (m.x == -INFINITY) continue;   // sees nothing of this piece
        const float w = ex2(m.x - M);
        L = fmaf(w, m.y, L);
        const float *src = a.acc + (pr + (size_t)k * CR) * D + lane * V;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(w, src[v], acc[v]);
    }
    const float r = 1.f / L;
    __half *dst = O + (((size_t)i * a.hq + j * hg + row % hg) * a.n_stride + row / hg) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t *>(dst + v) = ck_pack(acc[v] * r, acc[v + 1] * r);
}

template <int D, int NH>
cudaError_t launch_chunk(const KiviGeom &g, const KiviDev &dv, const __half *Q, const __half *K, const __half *V,
                         __half *O, ChunkArgs &a, int ctas, int maxrows, bool join, cudaStream_t st) {
    const size_t fixed = (size_t)NH * kCkRows * D * 2 + (size_t)2 * kCkStages * kCkKeys * D * 2;
    const size_t room = 226 * 1024 - fixed;
    a.rs = (int)(room / g.rec_bytes);
    if (a.rs > kCkMaxRaw) a.rs = kCkMaxRaw;
    if (a.rs < 2) return cudaErrorInvalidValue;
    const size_t smem = fixed + (size_t)a.rs * g.rec_bytes;
    cudaError_t e = cudaFuncSetAttribute(chunk_attn_kernel<D, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    chunk_attn_kernel<D, NH><<<ctas, 32 * (4 * NH + kCkDq + 3), smem, st>>>(g, dv, Q, K, V, O, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || !join) return e;
    chunk_join_kernel<D><<<dim3((maxrows + 7) / 8, g.h, g.b), 256, 0, st>>>(g, O, a, NH * kCkRows);
    return cudaGetLastError();
}

}  // namespace
