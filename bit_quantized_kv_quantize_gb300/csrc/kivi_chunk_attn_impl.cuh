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
// c of token r at byte c 1024 + r 16.  Warp w of the kCkDq takes the code
// chunks w, w + kCkDq, ...; a lane's half2 (two channels of one token) are
// the lanes t = 0..3 of one 16-byte chunk: 128 consecutive bytes a store.
template <int D, int KB>
__device__ __forceinline__ void dequant_keys(unsigned char *tile, const unsigned char *rec, int off_ksz, int lgG,
                                             int w) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const __half *ksz = reinterpret_cast<const __half *>(rec + off_ksz) + tq * (D / 4);
    unsigned char *dst = tile + gq * 16 + tq * 4;
    constexpr int JPC = KB == 2 ? 2 : 1;   // 16-channel steps a chunk of words covers
    for (int ch = w; ch < D * KB / 64; ch += kCkDq) {
        const uint4 w4 = *reinterpret_cast<const uint4 *>(rec + (size_t)ch * 512 + lane * 16);
#pragma unroll
        for (int jj = 0; jj < JPC; ++jj) {
            const int j = ch * JPC + jj;
            const uint32_t W[2][2] = {{KB == 2 && jj ? w4.z : w4.x, w4.y}, {KB == 2 ? (jj ? w4.w : w4.y) : w4.z, w4.w}};
#pragma unroll
            for (int qd = 0; qd < 4; ++qd) {   // 16 tokens share a group row
                const __half *row = ksz + (((16 * qd) >> lgG) * 2) * D + 4 * j;
                const uint2 s = *reinterpret_cast<const uint2 *>(row), z = *reinterpret_cast<const uint2 *>(row + D);
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int pos = 2 * qd + o;
                    const int wi = KB == 2 ? 0 : pos >> 2, r = KB == 2 ? pos : pos & 3;
                    const float off = slot_offset<KB, true>(r);
                    unsigned char *p = dst + (size_t)(2 * j) * (kCkKeys * 16) + pos * 128;
                    *reinterpret_cast<uint32_t *>(p) = ck_affine(unpack<KB, true>(W[0][wi], r), off, s.x, z.x);
                    *reinterpret_cast<uint32_t *>(p + kCkKeys * 16) =
                        ck_affine(unpack<KB, true>(W[1][wi], r), off, s.y, z.y);
                }
            }
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
    const uint32_t *words = reinterpret_cast<const uint32_t *>(rec + off_vc) + (size_t)w * (D * VB / 2);
    const __half *vsz = reinterpret_cast<const __half *>(rec + off_vsz) + (size_t)w * (2 * ngi * 16) + 4 * tq;
    uint32_t W[WL];
#pragma unroll
    for (int c = 0; c < WL / CS; ++c) {
        if (CS == 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(words + c * 128 + lane * 4);
            W[c * 4] = v.x;
            W[c * 4 + 1] = v.y;
            W[c * 4 + CS / 2] = v.z;
            W[c * 4 + CS - 1] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(words + c * 64 + lane * 2);
            W[c * 2] = v.x;
            W[c * 2 + 1] = v.y;
        }
    }
    unsigned char *dst = tile + (size_t)(2 * w) * (D * 16) + gq * 16 + tq * 4;
#pragma unroll
    for (int q = 0; q < D / 16; ++q) {   // 16 channels share a group row
        const int gi = (16 * q) >> lgG;
        const uint2 s = *reinterpret_cast<const uint2 *>(vsz + gi * 16);
        const uint2 z = *reinterpret_cast<const uint2 *>(vsz + (ngi + gi) * 16);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int ci = 2 * q + o, wi = ci / CPH, r = ci % CPH;
            const float off = slot_offset<VB, false>(r);
            *reinterpret_cast<uint32_t *>(dst + ci * 128) = ck_affine(unpack<VB, false>(W[wi], r), off, s.x, z.x);
            *reinterpret_cast<uint32_t *>(dst + D * 16 + ci * 128) =
                ck_affine(unpack<VB, false>(W[NWV + wi], r), off, s.y, z.y);
        }
    }
}

// Warps: 4 NH of softmax (thread tid owns row tid mod 128 of slot tid / 128,
// tensor-memory columns [256 slot, + 256): S / P buffers in 0-63 and 64-127,
// O from 128), kCkDq dequantizing, one issuing S = Q K^T, one O += P V.
// They meet on mbarriers (bounded waits): a tile's K^ / V^ written,
// read (MMA commits), S done, P written, P V done; records landed and read.
template <int D, int NH>
__global__ void __launch_bounds__(32 * (4 * NH + kCkDq + 2), 1)
    chunk_attn_kernel(KiviGeom g, KiviDev dv, const __half *__restrict__ Q, const __half *__restrict__ Kn,
                      const __half *__restrict__ Vn, __half *__restrict__ O, const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int QB = kCkRows * D * 2, TB = kCkKeys * D * 2;
    constexpr unsigned QLBO = kCkRows * 16, KLBO = kCkKeys * 16, VLBO = D * 16;
    constexpr int NSW = 4 * NH, CR = NH * kCkRows, TS = kCkStages;
    unsigned char *sQ = smem, *sK = sQ + NH * QB, *sV = sK + TS * TB, *sR = sV + TS * TB;
    __shared__ __align__(8) uint64_t bars[7 + 4 * TS + 2 * kCkMaxRaw];
    uint64_t *const bS = bars, *const bF = bars + 2, *const bP = bars + 4, *const bK = bars + 6, *const bV = bK + TS,
                    *const eK = bV + TS, *const eV = eK + TS, *const bR = eV + TS, *const eR = bR + kCkMaxRaw,
                    *const bX = eR + kCkMaxRaw;
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
        for (int k = 0; k < 7 + 4 * TS + 2 * kCkMaxRaw; ++k) {
            const bool written = k >= 6 && k < 6 + 2 * TS, read_raw = k >= 6 + 4 * TS + kCkMaxRaw;
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
    auto ph = [](int x, int m) { return (unsigned)(x / m) & 1u; };   // phase of use x of one of m stages

    if (warp == NSW + kCkDq) {
        // ---- S = Q K^T (lane 0) ----
        if (lane == 0) {
            constexpr uint32_t ID_S = tc_idesc_f16(kCkRows, kCkKeys, 0);
            int done = 0;
            for (int x = 0; x < nx; ++x) {
                // its K^ written, its S buffer free (P V of tile x - 2 read its weights there)
                ok = mbar_wait_ab(&bK[x % TS], ph(x, TS), abort) &&
                     (x < 2 || mbar_wait_ab(&bF[x & 1], ph(x - 2, 2), abort));
                if (!ok) break;
                tc_fence_after();
                const unsigned char *k = sK + (x % TS) * TB;
#pragma unroll
                for (int e = 0; e < NH; ++e)
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)
                        tc_mma_f16(taddr + 256 * e + 64 * (x & 1), tc_desc(sQ + e * QB + 2 * c * QLBO, QLBO, 128),
                                   tc_desc(k + 2 * c * KLBO, KLBO, 128), ID_S, c > 0);
                tc_commit(&bS[x & 1]);
                tc_commit(&eK[x % TS]);
                done = x + 1;
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            // every commit has landed before shared memory is given up (bounded)
            for (int x = max(0, done - 2); x < done; ++x) mbar_wait(&bS[x & 1], ph(x, 2));
            for (int x = max(0, done - TS); x < done; ++x) mbar_wait(&eK[x % TS], ph(x, TS));
        }
        __syncwarp();
    } else if (warp == NSW + kCkDq + 1) {
        // ---- O += P V (lane 0) ----
        if (lane == 0) {
            constexpr uint32_t ID_R = tc_idesc_f16(kCkRows, D, 1), ID_T = tc_idesc_f16(kCkRows, D, 0);
            int done = 0;
            for (int x = 0; x < nx; ++x) {
                ok = mbar_wait_ab(&bP[x & 1], ph(x, 2), abort) && mbar_wait_ab(&bV[x % TS], ph(x, TS), abort);
                if (!ok) break;
                tc_fence_after();
                const unsigned char *v = sV + (x % TS) * TB;
                const bool transposed = tile0(x) < Tqv;
#pragma unroll
                for (int e = 0; e < NH; ++e)
#pragma unroll
                    for (int c = 0; c < kCkKeys / 16; ++c)
                        tc_mma_f16_ta(taddr + 256 * e + 128, taddr + 256 * e + 64 * (x & 1) + 8 * c,
                                      transposed ? tc_desc(v + 2 * c * VLBO, VLBO, 128)
                                                 : tc_desc(v + 256 * c, 128, KLBO),
                                      transposed ? ID_T : ID_R, x > 0 || c > 0);
                tc_commit(&bF[x & 1]);
                tc_commit(&eV[x % TS]);
                done = x + 1;
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            for (int x = max(0, done - 2); x < done; ++x) mbar_wait(&bF[x & 1], ph(x, 2));
            for (int x = max(0, done - TS); x < done; ++x) mbar_wait(&eV[x % TS], ph(x, TS));
        }
        __syncwarp();
    } else if (warp >= NSW) {
        // ---- K^ and V^ tiles ----
        const int w = warp - NSW, dt = tid - 32 * NSW;   // dt: 0 .. 127
        const int lgG = __ffs(g.G) - 1;
        const int nraw = min(nx, max(0, bl.virt((max(Tqk, Tqv) + kCkKeys - 1) / kCkKeys) - x0));   // tiles with records
        const unsigned char *recs = dv.blk + rec_off(g, i, j, 0);
        const __half *kwin = dv.Kf + kf_slice(g, i, j), *vwin = dv.Vf + vf_slice(g, i, j);
        const __half *kch = Kn + ((size_t)i * g.h + j) * a.n_stride * D, *vch = Vn + ((size_t)i * g.h + j) * a.n_stride * D;
        auto issue_raw = [&](int x) {   // dt == 0
            uint64_t *bar = &bR[x % a.rs];
            mbar_expect_tx(bar, (unsigned)g.rec_bytes);
            bulk_g2s(sR + (size_t)(x % a.rs) * g.rec_bytes, recs + (size_t)(tile0(x) / kCkKeys) * g.rec_bytes,
                     (unsigned)g.rec_bytes, bar);
        };
        // the dequantizing warps meet (a bounded wait, unlike a named barrier)
        int meets = 0;
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bX);
            return __all_sync(0xffffffffu, mbar_wait_ab(bX, (unsigned)meets++ & 1u, abort)) != 0;
        };
        int issued = 0;
        if (dt == 0)
            for (; issued < min(nraw, a.rs); ++issued) issue_raw(issued);
        // fp16 rows: token tau's row in the window or the chunk (zero past the chunk)
        auto row16 = [&](const __half *win, int ring, const __half *chk, int tau, int c) {
            const __half *src = tau < T ? win + (size_t)(tau % ring) * D : chk + (size_t)(tau - T) * D;
            return tau < T + n ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        };
        constexpr int CPR = D / 8, RPT = kCkKeys * CPR / 128;   // 16-byte chunks a row; a thread's share of a tile
        for (int x = 0; x < nx; ++x) {
            const int tb = tile0(x), s = x % TS;
            unsigned char *kt = sK + s * TB, *vt = sV + s * TB;
            const bool raw = x < nraw;
            const bool kq = tb < Tqk, kall = tb + kCkKeys <= Tqk, vq = tb < Tqv, vall = tb + kCkKeys <= Tqv;
            // a record a few tiles ahead, into the stage that tile x - 1 has been read from
            if (x > 0 && x - 1 + a.rs < nraw) {
                if (dt == 0) {
                    ok = mbar_wait_ab(&eR[(x - 1) % a.rs], ph(x - 1, a.rs), abort);
                    if (ok) {
                        issue_raw(x - 1 + a.rs);
                        ++issued;
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            uint4 kr[RPT], vr[RPT];   // fp16 tiles: loads in flight before the waits
            if (!kq)
#pragma unroll
                for (int k = 0; k < RPT; ++k)
                    kr[k] = row16(kwin, g.R, kch, tb + (dt + 128 * k) / CPR, (dt + 128 * k) % CPR);
            if (!vq)
#pragma unroll
                for (int k = 0; k < RPT; ++k)
                    vr[k] = row16(vwin, g.R + 1, vch, tb + (dt + 128 * k) / CPR, (dt + 128 * k) % CPR);
            ok = (x < TS || mbar_wait_ab(&eK[s], ph(x - TS, TS), abort)) &&
                 (!raw || mbar_wait_ab(&bR[x % a.rs], ph(x, a.rs), abort));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const unsigned char *rec = sR + (size_t)(x % a.rs) * g.rec_bytes;
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
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bK[s]);
            ok = __all_sync(0xffffffffu, x < TS || mbar_wait_ab(&eV[s], ph(x - TS, TS), abort));
            if (!ok) break;
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
                mbar_arrive(&bV[s]);
                if (raw) mbar_arrive(&eR[x % a.rs]);
            }
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        if (dt == 0)   // every record copy has landed (bounded)
            for (int x = max(0, issued - a.rs); x < issued; ++x) mbar_wait(&bR[x % a.rs], ph(x, a.rs));
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
            ok = __all_sync(0xffffffffu, mbar_wait_ab(&bS[b], ph(x, 2), abort));
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
                ok = __all_sync(0xffffffffu, mbar_wait_ab(&bF[b ^ 1], ph(x - 1, 2), abort));
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
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_ab(&bF[(nx - 1) & 1], ph(nx - 1, 2), abort));
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
    chunk_attn_kernel<D, NH><<<ctas, 32 * (4 * NH + kCkDq + 2), smem, st>>>(g, dv, Q, K, V, O, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || !join) return e;
    chunk_join_kernel<D><<<dim3((maxrows + 7) / 8, g.h, g.b), 256, 0, st>>>(g, O, a, NH * kCkRows);
    return cudaGetLastError();
}

}  // namespace
