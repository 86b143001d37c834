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
// average like the values themselves (relative L2 error 3e-4 on even keys,
// up to 1.2e-3 where keys have channels 8 times the others; an fp16 output
// alone rounds by 2e-4).
//
// Pipeline.  A slot has two S buffers of 64 columns (P over the first 32) and
// O.  One warp issues the S MMAs, up to two tiles ahead (once the P V that
// reads a buffer's weights is done), another the P V MMAs, so that a wait of
// one does not hold the other back; slots wait for their own work only.  (One 128-column buffer a slot, S
// following P V, makes the softmax, P V and S of a slot a serial chain:
// 5150 against 4400 cycles a 128-token tile pair, measured.)
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
#include <cuda_fp16.h>

#include "kivi_async.cuh"
#include "kivi_chunk.cuh"
#include "kivi_internal.cuh"
#include "kivi_mma.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_tma.cuh"
#include "kivi_unpack.cuh"

namespace {

constexpr int kCkRows = 128;     // rows of a slot
constexpr int kCkKeys = KIVI_KBLK;   // tokens of a tile
constexpr int kCkStages = 3;     // K^ tiles, and V^ tiles, in flight
constexpr int kCkMaxRaw = 8;     // records in flight
constexpr int kCkDq = 4;         // dequantizing warps
constexpr int kCkOut = 8 * 32 * 64;   // a softmax warp's 32 rows x 32 columns of the output
constexpr int kCkThreads = 32 * (8 + kCkDq + 3);
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ uint32_t ck_pack(float lo, float hi) {
    return h2u(__floats2half2_rn(lo, hi));
}
// s code + z of two values, the code from off + code (exact)
__device__ __forceinline__ uint32_t ck_affine(uint32_t x, float off, uint32_t s, uint32_t z) {
    return h2u(__hfma2(__hsub2(u2h(x), __float2half2_rn(off)), u2h(s), u2h(z)));
}


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

// A CTA's share of one row tile.
struct CkSeg {
    int i, j, m;     // sequence, kv head, row tile
    int T, n;        // cached tokens, chunk tokens
    int row0, nrows; // first row, rows of (i, j)
    int nt;          // its key tiles
    int x0, nx;      // the CTA's of them
    BlockList bl;
    // first token of the CTA's tile x
    __device__ __forceinline__ int key0(int x) const { return bl.phys(x0 + x) * kCkKeys; }
};

// Walks a CTA's unit range [u, u1): every warp runs the same walk.
struct CkWalk {
    long long u, u1;
    int i, m, j;     // the row tile holding u ...
    int o;           // ... and u's offset in it
    __device__ __forceinline__ int weight(const KiviGeom &g, const ChunkArgs &a) const {
        return kCkLead + chunk_tiles(a, i, m, a.hq / g.h);
    }
    __device__ __forceinline__ void start(const KiviGeom &g, const ChunkArgs &a, int c, int C) {
        const long long U = a.ustart[g.b];
        u = (long long)c * U / C;
        u1 = (long long)(c + 1) * U / C;
        int lo = 0;
        for (int hi = g.b; hi - lo > 1;) {
            const int mid = (lo + hi) >> 1;
            if (a.ustart[mid] <= u) lo = mid; else hi = mid;
        }
        i = lo;
        const int hg = a.hq / g.h, lane = threadIdx.x & 31, mt = chunk_row_tiles(a.n[i], hg);
        long long rem = u - a.ustart[i];
        for (m = 0;; m += 32) {   // 32 row tiles of every head at a time
            const long long w = m + lane < mt ? (long long)g.h * (kCkLead + chunk_tiles(a, i, m + lane, hg)) : 0;
            long long e = w;   // inclusive prefix
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(kFull, e, d);
                if (lane >= d) e += y;
            }
            const unsigned past = __ballot_sync(kFull, e > rem);
            if (past || m + 32 >= mt) {
                const int l = past ? __ffs(past) - 1 : 31;
                rem -= __shfl_sync(kFull, e - w, l);
                m += l;
                break;
            }
            rem -= __shfl_sync(kFull, e, 31);
        }
        const int w = weight(g, a);
        j = (int)(rem / w);
        o = (int)(rem % w);
    }
    // the next segment with tiles; false at the range's end
    __device__ __forceinline__ bool next(const KiviGeom &g, const ChunkArgs &a, CkSeg &s) {
        const int hg = a.hq / g.h;
        while (u < u1) {
            const int w = weight(g, a), o1 = (int)min((long long)w, o + (u1 - u));
            const int x0 = max(o - kCkLead, 0), x1 = max(o1 - kCkLead, 0);
            if (x1 > x0) {
                s.i = i;
                s.j = j;
                s.m = m;
                s.T = a.T[i];
                s.n = a.n[i];
                s.row0 = m * kCkTileRows;
                s.nrows = s.n * hg;
                s.nt = w - kCkLead;
                s.x0 = x0;
                s.nx = x1 - x0;
                s.bl = visible_blocks(a.vis, s.T + s.row0 / hg);
            }
            u += o1 - o;
            o = 0;
            if (o1 == w && ++j == g.h) {
                j = 0;
                if (++m == chunk_row_tiles(a.n[i], hg)) {
                    m = 0;
                    do ++i; while (i < g.b && a.n[i] == 0);
                }
            }
            if (x1 > x0) return true;
        }
        return false;
    }
};

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
    for (int x = 0; x < n; ++x, ++tiles) {
        bool ok = (tiles < kCkStages || mbar_wait_ab(&eK[t.s], t.p ^ 1u, abort)) && mbar_wait_ab(&bR[r.s], r.p, abort);
        if (!__all_sync(kFull, ok)) return false;
        const unsigned char *rec = sR + (size_t)r.s * g.rec_bytes;
        dequant_keys<D, KB>(sK + t.s * TB, rec, g.off_ksz, lgG, w);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bK[t.s]);
        ok = tiles < kCkStages || mbar_wait_ab(&eV[t.s], t.p ^ 1u, abort);
        if (!__all_sync(kFull, ok)) return false;
        dequant_values<D, VB>(sV + t.s * TB, rec, g.off_vc, g.off_vsz, lgG, w);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bV[t.s]);
            mbar_arrive(&eR[r.s]);
        }
        t.next(kCkStages);
        r.next(rs);
    }
    return true;
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
// tensor-memory columns [256 slot, + 256): S / P buffers in 0-63 and 64-127,
// O from 128); 8-11: dequantizing; 12: S = Q K^T; 13: O += P V; 14: record copies.  They
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
    // a meeting, K and V tiles written, records read; 1: the others
    constexpr int N4 = 7 + 2 * KS + kCkMaxRaw, NB = N4 + 8 + 2 * KS + kCkMaxRaw;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bQ = bars, *const bP = bars + 2, *const bX = bars + 6, *const bK = bars + 7, *const bV = bK + KS,
                    *const eR = bV + KS, *const bS = bars + N4, *const bF = bS + 4, *const eK = bF + 4,
                    *const eV = eK + KS, *const bR = eV + KS;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;   // a wait ran out: every warp stops
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = a.hq / g.h;
    const bool qtma = kCkRows % hg == 0;   // Q's row tiles are boxes of its array
    if (tid < NB) {
        mbar_init(&bars[tid], tid < N4 && !(qtma && tid < 2) ? 4 : 1);
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
    walk.start(g, a, blockIdx.x, gridDim.x);
    CkSeg sg = {};
    // the segment's first tiles have a record: how many
    auto raw_tiles = [&](int Tq) {
        return max(0, min(sg.x0 + sg.nx, sg.bl.virt((Tq + kCkKeys - 1) / kCkKeys)) - sg.x0);
    };

    if (warp == 8 + kCkDq) {
        // ---- S = Q K^T (lane 0 issues) ----
        constexpr uint32_t ID_S = tc_idesc_f16(kCkRows, kCkKeys, 0);
        CkRing tk;
        int nk = 0;             // K tiles read
        int cs[2] = {0, 0};     // S of each slot
        unsigned qph[2] = {0, 0};
        while (walk.next(g, a, sg)) {
            if (lane == 0) {
                const int slots = sg.nrows - sg.row0 > kCkRows ? 2 : 1;
                if (qtma) {   // this segment's Q, once the last one's S is done
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e >= slots || !ok) continue;
                        ok = cs[e] == 0 || mbar_wait_ab(&bS[2 * e + ((cs[e] - 1) & 1)], (unsigned)((cs[e] - 1) >> 1) & 1u, abort);
                        if (ok) tma_rows(sQ + e * QB, &tmQ, (sg.row0 + e * kCkRows) / hg, sg.i * g.h + sg.j, &bQ[e], QB);
                    }
                }
                for (int x = 0; x < sg.nx && ok; ++x) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e >= slots || !ok) continue;
                        // its Q and K written, its S buffer free (P V of the slot's
                        // last tile but one, in this segment or before, read its
                        // weights there)
                        const int b = cs[e] & 1;
                        ok = (x > 0 || mbar_wait_ab(&bQ[e], qph[e], abort)) &&
                             (e > 0 || mbar_wait_ab(&bK[tk.s], tk.p, abort)) &&
                             (cs[e] < 2 || mbar_wait_ab(&bF[2 * e + b], (unsigned)((cs[e] >> 1) + 1) & 1u, abort));
                        if (!ok) continue;
                        if (x == 0) qph[e] ^= 1u;
                        ++cs[e];
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < D / 16; ++c)
                            tc_mma_f16(taddr + 256 * e + 64 * b, tc_desc(sQ + e * QB + 2 * c * QLBO, QLBO, 128),
                                       tc_desc(sK + tk.s * TB + 2 * c * KLBO, KLBO, 128), ID_S, c > 0);
                        tc_commit(&bS[2 * e + b]);
                        if (e == slots - 1) {
                            tc_commit(&eK[tk.s]);
                            tk.next(KS);
                            ++nk;
                        }
                    }
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
            // every commit has landed before shared memory is given up
            // (bounded; a phase already seen returns at once)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                for (int y = max(0, cs[e] - 2); y < cs[e]; ++y) mbar_wait(&bS[2 * e + (y & 1)], (unsigned)(y >> 1) & 1u);
            for (int y = max(0, nk - KS); y < nk; ++y) mbar_wait(&eK[y % KS], (unsigned)(y / KS) & 1u);
        }
        __syncwarp();
    } else if (warp == 8 + kCkDq + 1) {
        // ---- O += P V (lane 0 issues) ----
        constexpr uint32_t ID_R = tc_idesc_f16(kCkRows, D, 1), ID_T = tc_idesc_f16(kCkRows, D, 0);
        CkRing tv;
        int nv = 0;             // V tiles read
        int cp[2] = {0, 0};     // P V of each slot
        while (walk.next(g, a, sg)) {
            if (lane == 0) {
                const int slots = sg.nrows - sg.row0 > kCkRows ? 2 : 1;
                const int Tqv = a.Tqv[sg.i];
                for (int x = 0; x < sg.nx && ok; ++x) {
                    const bool transposed = sg.key0(x) < Tqv;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e >= slots || !ok) continue;
                        const int b = cp[e] & 1;
                        ok = mbar_wait_ab(&bP[2 * e + b], (unsigned)(cp[e] >> 1) & 1u, abort) &&
                             (e > 0 || mbar_wait_ab(&bV[tv.s], tv.p, abort));
                        if (!ok) continue;
                        ++cp[e];
                        tc_fence_after();
                        const unsigned char *v = sV + tv.s * TB;
                        const uint32_t tO = taddr + 256 * e + 128, tP = taddr + 256 * e + 64 * b;
#pragma unroll
                        for (int c = 0; c < kCkKeys / 16; ++c)
                            tc_mma_f16_ta(tO, tP + 8 * c,
                                          transposed ? tc_desc(v + 2 * c * VLBO, VLBO, 128) : tc_desc(v + 256 * c, 128, KLBO),
                                          transposed ? ID_T : ID_R, x > 0 || c > 0);
                        tc_commit(&bF[2 * e + b]);
                        if (e == slots - 1) {
                            tc_commit(&eV[tv.s]);
                            tv.next(KS);
                            ++nv;
                        }
                    }
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
#pragma unroll
            for (int e = 0; e < 2; ++e)
                for (int y = max(0, cp[e] - 2); y < cp[e]; ++y) mbar_wait(&bF[2 * e + (y & 1)], (unsigned)(y >> 1) & 1u);
            for (int y = max(0, nv - KS); y < nv; ++y) mbar_wait(&eV[y % KS], (unsigned)(y / KS) & 1u);
        }
        __syncwarp();
    } else if (warp == 8 + kCkDq + 2) {
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
        int tiles = 0, meets = 0;
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
            for (int x = npk; x < sg.nx && ok; ++x, ++tiles, t.next(KS)) {
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
                    if (g.kbits == 2) dequant_keys<D, 2>(kt, rec, g.off_ksz, lgG, w);
                    else dequant_keys<D, 4>(kt, rec, g.off_ksz, lgG, w);
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
                ok = __all_sync(kFull, tiles < KS || mbar_wait_ab(&eV[t.s], t.p ^ 1u, abort));
                if (!ok) break;
                if (vq) {
                    if (g.vbits == 2) dequant_values<D, 2>(vt, rec, g.off_vc, g.off_vsz, lgG, w);
                    else dequant_values<D, 4>(vt, rec, g.off_vc, g.off_vsz, lgG, w);
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
        if (!ok) {
            if (lane == 0) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            // a TMA copy may be in flight: the bounded waits outlast it
            mbar_wait(&bK[t.s], t.p);
            mbar_wait(&bV[t.s], t.p);
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
                        const int rw = min(srow + qr(k0 + k), sg.nrows - 1);
                        v[k] = *reinterpret_cast<const uint4 *>(
                            Q + (((size_t)sg.i * a.hq + sg.j * hg + rw % hg) * a.n_stride + rw / hg) * D + 8 * qc(k0 + k));
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
            const int pos = sg.T + row / hg, ps0 = sg.T + srow / hg, ps1 = sg.T + (srow + kCkRows - 1) / hg;
            const int lo = W > 0 ? pos - W : -1;   // tokens [sinks, lo] are hidden
            float mref = -INFINITY, lsum = 0.f;    // the row's reference maximum (raw score units) and weight sum
            for (int x = 0; x < sg.nx; ++x, ++cnt) {
                const int b = cnt & 1, key0 = sg.key0(x);
                ok = __all_sync(kFull, mbar_wait_ab(&bS[2 * slot + b], (unsigned)(cnt >> 1) & 1u, abort));
                if (!ok) break;
                tc_fence_after();
                uint32_t r[2][32];   // this row's 64 scores
                tc_ld32(tS + 64 * b, r[0]);
                tc_ld32(tS + 64 * b + 32, r[1]);
                tc_wait_ld();
                if (key0 + kCkKeys - 1 > ps0 || (W > 0 && key0 <= ps1 - W && key0 + kCkKeys > sinks)) {
                    // some row of the slot does not see the whole tile
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        const int key = key0 + c;
                        if (key > pos || (key <= lo && key >= sinks)) r[c >> 5][c & 31] = 0xff800000u;
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
                const bool grow = mx != -INFINITY && (mref == -INFINITY || (mx - mref) * sl2 > 8.f);
                const float alpha = grow && mref != -INFINITY ? ex2((mref - mx) * sl2) : 1.f;
                if (grow) mref = mx;
                const float ms = mref == -INFINITY ? 0.f : mref * sl2;   // (nothing seen yet: weights 0)
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
                tc_st32(tS + 64 * b, pw);   // P over the first 32 columns of its S buffer
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bP[2 * slot + b]);
            }
            // the last P V (the one before it ended before its S, which was waited
            // for, was issued, or is waited for first)
            for (int y = max(cnt - 2, cnt - sg.nx); y < cnt && ok; ++y)
                ok = __all_sync(kFull, mbar_wait_ab(&bF[2 * slot + (y & 1)], (unsigned)(y >> 1) & 1u, abort));
            if (!ok) break;
            tc_fence_after();
            if (sg.nx < sg.nt) {   // this CTA's partial of the row
                const size_t pr = (size_t)(2 * blockIdx.x + (sg.x0 == 0 ? 1 : 0)) * kCkTileRows + slot * kCkRows + rr;
                if (in) reinterpret_cast<float2 *>(a.ml)[pr] = make_float2(mref * sl2, lsum);
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
                    const int rw = min(row32 + 8 * k + q8, sg.nrows - 1);
                    orow[k] = (((size_t)sg.i * a.hq + sg.j * hg + rw % hg) * a.n_stride + rw / hg) * D + 8 * c4;
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
    if (warp == 0) tc_dealloc(taddr, 512);
}

// Joins the partials of the row tiles that CTA boundaries cut, a block per
// cut row tile and 32 of its rows (a warp takes rows w, w + 8, ...): weights
// 2^(m_k - M), M the largest m.  Block x finds its row tile from the boundary
// before CTA x / 8 + 1: the tile's first such boundary owns it.
template <int D>
__global__ void __launch_bounds__(256)
    chunk_join_kernel(KiviGeom g, __half *__restrict__ O, const __grid_constant__ ChunkArgs a, int ctas) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hg = a.hq / g.h, c = blockIdx.x / (kCkTileRows / 32) + 1;
    CkWalk walk;
    walk.start(g, a, c, ctas);
    if (walk.o <= kCkLead) return;   // CTA c starts with a row tile of its own
    const long long U = a.ustart[g.b], P = walk.u - walk.o;
    const int w = walk.weight(g, a), i = walk.i, j = walk.j;
    auto cta_of = [&](long long u) { return (int)(((u + 1) * ctas - 1) / U); };
    const int c0 = cta_of(P + kCkLead), c1 = cta_of(P + w - 1);   // those with its tiles
    if (c != c0 + 1) return;         // an earlier boundary owns the row tile
    // CTA c0 holds its first tile and runs into it (slot 2 c + 1), the others
    // start in it (slot 2 c)
    const float2 *ml = reinterpret_cast<const float2 *>(a.ml);
    const int nrows = min(a.n[i] * hg - walk.m * kCkTileRows, kCkTileRows);
    for (int r = (blockIdx.x % (kCkTileRows / 32)) * 32 + warp; r < min(nrows, (int)(blockIdx.x % (kCkTileRows / 32)) * 32 + 32);
         r += 8) {
        auto part = [&](int k) { return (size_t)(2 * k + (k == c0 ? 1 : 0)) * kCkTileRows + r; };
        float M = -INFINITY;
        for (int k = c0 + lane; k <= c1; k += 32) M = fmaxf(M, ml[part(k)].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
        float L = 0.f, acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
        for (int k = c0; k <= c1; ++k) {
            const float2 x = ml[part(k)];
            const float wt = x.x == -INFINITY ? 0.f : ex2(x.x - M);   // (sees nothing of this share)
            L = fmaf(wt, x.y, L);
            const float *src = a.acc + part(k) * D + lane * V;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(wt, src[v], acc[v]);
        }
        const float inv = 1.f / L;
        const int row = walk.m * kCkTileRows + r;
        __half *dst = O + (((size_t)i * a.hq + j * hg + row % hg) * a.n_stride + row / hg) * D + lane * V;
#pragma unroll
        for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t *>(dst + v) = ck_pack(acc[v] * inv, acc[v + 1] * inv);
    }
}

}  // namespace
