// kivi_latent_attn.cu -- latent attention in its absorbed form: new tokens over
// the quantized latent cache and over themselves, on the 5th-generation tensor
// cores.
//
// Mathematics.  With q = [Wk_h^T qn ; qr] (r + 64 channels) and a token's
// row t_s = [c_s ; kr_s], head h of the token at position p has
//   out = sum_s softmax_s(scale q . t_s) c_s   over s <= p:
// one key and value row a token for every head.  So the rows (token, head) of a
// sequence are one list, cut into row tiles of RN = 64 or 32, and a tile of 128
// tokens, restored once to fp16 in shared memory, is the A operand of both
//   S^T [128 tokens x RN rows] = T Q^T      (r + 64 deep)
// and, read along its other axis,
//   O^T [r x RN rows] += C^T P^T            (128 deep, r / 128 MMAs of 128 rows).
//
// Bound: shared memory's bandwidth.  An MMA of 128 x 64 x 16 reads 6 KB of it (48
// cycles, for 32 of the tensor cores'); with the restoring's stores a tile of r =
// 512 moves 570 KB, 4450 cycles of it, and takes 6500: with one tile in shared
// memory its steps follow one another (waits for the last parts and the end of S^T
// 1800 cycles, softmax 1200, O^T's first part 1000), and only the restoring, 2500,
// runs beside the products.  8 x 32k 4-bit tokens of 128 heads (73 GFLOP): 142 us
// and 8 for the join; 64 ragged sequences of 4k, 16 heads: 35 in all; 1024 tokens of
// 16 heads over 8000: 515.
// 64 rows are what tensor memory holds: r x 64 sums take r / 2 of its 512 columns.
// (S with the 64 rows on the M side and tiles of 64 tokens, two of which fit, took as
// long an MMA, 49 cycles measured, for half of the tokens: 220 us over the 32k.)
// Where row tiles of 32 are no more than those of 64, as in a step of up to 32
// heads, an MMA takes 40 cycles and a softmax 700: the 64 ragged sequences' attention
// 35 us for 39.
//
// A thread of the softmax has one token and a quarter of the rows, so a row's maximum over
// the tile is spread over threads.  It is not formed a tile: weights are taken
// against the row's reference, and only when some score lies more than 2^8 above
// it (one vote a tile) are the maxima formed, the references raised, O^T's columns
// and the sums rescaled, as in the chunk attention's kernel for few rows.
//
// Rounding.  A restored latent vector (scale code + zero), the weights and the
// query enter the products in fp16 (2^-11 relative each); sums in fp32.
//
// Work split (as the chunk attention's): the tiles of all row tiles end to end,
// each CTA an equal share, cut row tiles joined from partials.
#include "kivi_chunk_tiles.cuh"
#include "kivi_latent.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_tma.cuh"

namespace {

// Warps that restore tiles and take their softmax: with two more for the MMAs and
// copies, 18 warps of 96 registers.  (8 of 168: 160 us over the 32k for 150.  What is
// live over a tile has to fit: spills go to L2 where shared memory takes all of the
// first-level cache, and calls of other functions in the loop spill, 180 to 275 us.)
constexpr int kLaWork = 16;
constexpr int kLaThreads = 32 * (kLaWork + 2);
// Tiles that stand for a row tile's fixed cost, 14,000 cycles and a cut one's partials
// (2: as long; 1 and 4: 3 % longer).
constexpr int kLaLead = 3;
__host__ __device__ constexpr int la_cols(int rows) { return rows / (kLaWork / 4); }   // rows of a thread in the softmax
constexpr unsigned kLaCS = kLatTok * 128;    // bytes of 64 channels of a tile
// tiles in shared memory (of r = 512 one fits; it is refilled in parts)
__host__ __device__ constexpr int la_stages(int r) { return r == 512 ? 1 : 2; }
__host__ __device__ constexpr int la_tile(int r) { return (r + kLatRope) / 64 * (int)kLaCS; }
__host__ __device__ constexpr size_t la_smem(int r, int rows) {
    return (size_t)la_stages(r) * la_tile(r) + (r + kLatRope) / 64 * rows * 128 + 1024;
}
constexpr float kLaUnset = 1e30f;   // s_ref of a row that has seen nothing

// whether any of the working warps says v (all come here every tile)
__device__ __forceinline__ bool la_any(bool v) {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "n"(32 * kLaWork)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void la_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kLaWork) : "memory"); }
__device__ __forceinline__ float la_redux_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// 16 bytes of codes of a token (128 / BITS channels) to their chunks of its row
// (at: the first one's place): sz the scales and zeros of their halves (4 bits: of
// all).
template <int BITS>
__device__ __forceinline__ void la_restore(unsigned char *tile, unsigned at, const uint4 &v, const uint32_t *sz) {
    constexpr int PW = 32 / BITS, CW = 4 * PW, NG = CW / 32;   // channels a 32-bit word, the 16 bytes
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < CW / 8; ++c) {   // 8 channels: one 16-byte chunk
        const __half2 p = u2h(sz[c * NG / (CW / 8)]);
        const uint32_t s = h2u(__low2half2(p)), z = h2u(__high2half2(p));
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int f = (8 * c % PW) / 2 + k;   // field of the word's halves
            o[k] = ck_affine(unpack<BITS, false>(w[8 * c / PW], f), slot_offset<BITS, false>(f), s, z);
        }
        *reinterpret_cast<uint4 *>(tile + (at ^ (c << 4))) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// A warp's part of a tile: units of one 16-byte word of codes (CW channels) of 32
// tokens, a lane each.  Unit k is word x0 + WX k (x0: warp / 4); PU of them are of a
// part of 128 channels, or the words that the warps have at a time span SPAN parts.
template <int RD, int BITS>
struct LaUnits {
    static constexpr int WX = kLaWork / 4;   // words at a time
    static constexpr int CW = 128 / BITS, NU = RD / CW / WX, NG = CW / 32, SPAN = WX * CW > 128 ? WX * CW / 128 : 1;
    static constexpr int PU = WX * CW > 128 ? 1 : 128 / CW / WX;
    uint4 w[NU];
    uint32_t sz[NU][NG];
    // p: unit 0's codes in the record; z: the record's scales and zeros of the
    // warp's token; ch: unit 0's first channel
    __device__ __forceinline__ void load(const unsigned char *p, const unsigned char *z, int ch, int lgG) {
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            w[k] = *reinterpret_cast<const uint4 *>(p + k * (WX * kLatTok * 16));
#pragma unroll
            for (int q = 0; q < NG; ++q)
                sz[k][q] = *reinterpret_cast<const uint32_t *>(z + ((ch + WX * CW * k + 32 * q) >> lgG) * (kLatTok * 4));
        }
    }
};

// What a tile holds, and who fills it: codes only (restored by the working warps),
// or fp16 rows (copied).
struct LaTile {
    int tb;
    bool packed;   // codes only
    bool block;    // a whole block of the ring
    bool keys;     // the rotary keys are a whole block of the cache
    __device__ __forceinline__ LaTile(int tb, int T, int Tq)
        : tb(tb), packed(tb + kLatTok <= Tq), block(!packed && tb + kLatTok <= T), keys(tb + kLatTok <= T) {}
};

// a thread's columns of a row tile
__device__ __forceinline__ void la_ld(uint32_t t, uint32_t (&r)[8]) { tc_ld8(t, r); }
__device__ __forceinline__ void la_ld(uint32_t t, uint32_t (&r)[16]) { tc_ld16(t, r); }
__device__ __forceinline__ void la_st(uint32_t t, const uint32_t (&r)[16]) { tc_st16(t, r); }
__device__ __forceinline__ void la_st(uint32_t t, const uint32_t (&r)[8]) { tc_st8(t, r); }

// A raise: the rows' maxima over the tile (tS: this warp's scores of its rows, of
// which those c < lim do not see the token), the references of the rows that grew by
// more than 2^8, and their factors.  Called by every working warp.
template <int RN>
__device__ __forceinline__ void la_raise(uint32_t tS, float sl2, int lim, float *s_ref, float *s_al, float (*s_red)[kLatRows]) {
    constexpr int CN = la_cols(RN);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t r[CN];
    la_ld(tS, r);
    tc_wait_ld();
#pragma unroll
    for (int c = 0; c < CN; ++c) {
        const float m = la_redux_max(c < lim ? -INFINITY : __uint_as_float(r[c]) * sl2);
        if (lane == 0) s_red[warp & 3][CN * (warp >> 2) + c] = m;
    }
    la_sync();
    const int t = threadIdx.x;
    if (t < RN) {
        const float m = fmaxf(fmaxf(s_red[0][t], s_red[1][t]), fmaxf(s_red[2][t], s_red[3][t]));
        const float old = s_ref[t];
        const bool grow = m != -INFINITY && m + old > kCkLift + kCkLag;
        s_al[t] = grow && old != kLaUnset ? ex2((kCkLift - m) - old) : 1.f;
        if (grow) s_ref[t] = kCkLift - m;
    }
    la_sync();
}
// A warp's columns of O^T times the rows' factors, NM times (tO: this warp's lanes)
template <int RN, int NM>
__device__ __forceinline__ void la_rescale(uint32_t tO, const float *al) {
    constexpr int CN = la_cols(RN);
#pragma unroll 1
    for (int m = 0; m < NM; ++m) {
        uint32_t o[CN];
        la_ld(tO + RN * m, o);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < CN; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * al[c]);
        la_st(tO + RN * m, o);
    }
    tc_wait_st();
}

// One thread's weights of its token against the references of its rows, from
// the scores at tS: into its row of P (sP: the shared-memory address of its first
// chunk), their sums from tL0 (first: none yet) to tL1.  Rows c < lim do not see the
// token.  The largest log2 weight.
template <int RN>
__device__ __forceinline__ float la_weights(uint32_t tS, uint32_t tL0, uint32_t tL1, bool first, unsigned sP,
                                            const float *refs, float sl2, int lim) {
    constexpr int CN = la_cols(RN);
    float up = -INFINITY;
    uint32_t r[CN], l[CN];
    la_ld(tS, r);
    if (!first) la_ld(tL0, l);
    tc_wait_ld();
    if (first)
#pragma unroll
        for (int c = 0; c < CN; ++c) l[c] = 0u;
#pragma unroll
    for (int c = 0; c < CN; c += 8) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            const float4 ref = *reinterpret_cast<const float4 *>(refs + c + k);
            y[k] = fmaf(__uint_as_float(r[c + k]), sl2, ref.x);
            y[k + 1] = fmaf(__uint_as_float(r[c + k + 1]), sl2, ref.y);
            y[k + 2] = fmaf(__uint_as_float(r[c + k + 2]), sl2, ref.z);
            y[k + 3] = fmaf(__uint_as_float(r[c + k + 3]), sl2, ref.w);
        }
        if (lim > c)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k < lim) y[k] = -INFINITY;
        uint32_t pw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            up = fmaxf(up, fmaxf(y[2 * k], y[2 * k + 1]));
            const float y0 = ex2(y[2 * k]), y1 = ex2(y[2 * k + 1]);
            l[c + 2 * k] = __float_as_uint(__uint_as_float(l[c + 2 * k]) + y0);
            l[c + 2 * k + 1] = __float_as_uint(__uint_as_float(l[c + 2 * k + 1]) + y1);
            pw[k] = ck_pack(y0, y1);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sP ^ ((c / 8) << 4)), "r"(pw[0]), "r"(pw[1]), "r"(pw[2]),
                     "r"(pw[3])
                     : "memory");
    }
    la_st(tL1, l);
    tc_wait_st();
    fence_proxy_async();
    tc_fence_before();
    return up;
}

// Warps 0-15: restoring tiles, softmax and output (of r = 512 one tile fits, so that
// the two never run at once); 16: S^T and O^T; 17: copies (rotary keys, whole fp16
// tiles).  They meet on mbarriers only (bounded
// waits).  A tile is filled, and given back, in parts of 128 channels: S^T of the
// next tile begins with its first part while O^T still reads the others.  Tensor
// memory: two S^T buffers of RN columns, O^T, two buffers of the weights' sums.
// Shared memory: tiles, then Q, both in lat_at's layout.  The weights (a row of RN a
// token) take the place of the tile's rotary keys, which only S^T reads.
template <int RD, int BITS, int RN>
__global__ void __launch_bounds__(kLaThreads, 1)
    latent_attn_kernel(const __grid_constant__ LatentGeom g, const __grid_constant__ LatentDev dv,
                       const __half *Q, const __half *Qr, const __half *Cn, const __half *Kn, __half *O, const __grid_constant__ CUtensorMap tmC,
                       const __grid_constant__ CUtensorMap tmK, float sl2, const __grid_constant__ ChunkArgs a) {
    extern __shared__ unsigned char raw[];
    unsigned char *const smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    constexpr int KS = la_stages(RD), TB = la_tile(RD), NM = RD / 128;
    constexpr unsigned CB = RD / 64 * kLaCS, RB = kLatRope / 64 * kLaCS;   // bytes of a tile's c, and kr
    static_assert(RB >= RN * kLatTok * 2, "the weights fit in the rotary keys' place");
    constexpr int CN = la_cols(RN);
    constexpr unsigned QS = RN * 128;   // bytes of 64 channels of Q
    constexpr int OC = 2 * RN;   // first column of O^T
    unsigned char *sC = smem, *sQ = sC + KS * TB;
    using Units = LaUnits<RD, BITS>;
    // counts the working warps: Q, parts of a tile restored [stage][part]; 1: the
    // others (bR, bK: parts and rotary keys copied; each part waits for both.  bF: O^T
    // done, two in turn, as it may be two tiles behind the softmax)
    constexpr int N8 = 1 + KS * NM, NB = N8 + 2 * KS * NM + KS + 8;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bQ = bars, *const bC = bars + 1, *const eC = bars + N8, *const bR = eC + KS * NM,
                    *const bK = bR + KS * NM, *const bP = bK + KS, *const bS = bP + 2, *const bF = bS + 2, *const bE = bF + 2, *const bX = bE + 1;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;
    __shared__ __align__(16) float s_ref[kLatRows];   // the lift less each row's reference (log2 units)
    __shared__ __align__(16) float s_al[kLatRows];    // a raise's factors; 1 / sum of each row
    __shared__ float s_red[4][kLatRows];              // per 32 tokens: maxima, or sums
    __shared__ CkSeg s_seg;                           // for the segment's end (out of the tile loop's registers)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = a.hg;
    if (tid < NB) {
        mbar_init(&bars[tid], tid == 0 ? kLaWork : tid < N8 ? kLaWork / Units::SPAN : 1);
        fence_mbar_init();
    }
    if (tid == 0) s_abort = 0;
    if (warp == 0) tc_alloc(&s_taddr, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    kivi_after_previous<false>();
    const uint32_t taddr = s_taddr;
    const volatile int *abort = &s_abort;
    bool ok = true;
    KiviGeom kg;   // (the walk reads b and h)
    kg.b = g.b;
    kg.h = 1;
    CkWalk<kLaLead> walk;
    walk.start(a, blockIdx.x);
    CkSeg sg = {};
    constexpr int WS = kLaWork;

    if (warp == WS) {
        // ---- S^T = T Q^T of tile x, then O^T += C^T P^T of tile x - (KS - 1) ----
        constexpr uint32_t IDS = tc_idesc_f16(kLatTok, RN, 0);
        constexpr uint32_t IDO = tc_idesc_f16_at(128, RN) | (1u << 16);   // both MN-major
        CkRing t, u;
        int cs = 0, co = 0;   // S^T, O^T so far
        unsigned qph = 0;
        const uint64_t dq = tc_desc_sw(sQ, 16, 1024), ds = tc_desc_sw(sC, 16, 1024);
        const uint64_t dc = tc_desc_sw(sC, kLaCS, 1024), dp = tc_desc_sw(sC + CB, 16, 1024);
        while (ok && walk.next(kg, a, sg)) {
            const int nx = __reduce_max_sync(kFull, sg.nx);
            for (int x = 0; x < nx + KS - 1; ++x) {
                if (x < nx) {
                    const int b = cs & 1;
                    // (the buffer's last scores are read: with one tile O^T waited for their
                    // weights, with two that of the last but one did)
                    ok = x > 0 || mbar_wait_ab(bQ, qph, abort);
                    const uint64_t d = ds + (uint32_t)(t.s * (TB >> 4));
                    auto part_in = [&](int m, auto wait) {
                        return m < NM ? wait(&bC[t.s * NM + m]) && wait(&bR[t.s * NM + m]) : wait(&bK[t.s]);
                    };
                    bool in = false;   // the part is in (polled while the last one's products are issued)
#pragma unroll
                    for (int m = 0; m <= NM; ++m) {   // its parts, then the rotary keys
                        ok = __all_sync(kFull, ok && (in || part_in(m, [&](uint64_t *bar) { return mbar_wait_ab(bar, t.p, abort); })));
                        if (!ok) break;
                        in = m < NM && part_in(m + 1, [&](uint64_t *bar) { return mbar_test(bar, t.p); });
                        tc_fence_after();
                        const uint64_t qm = dq + (uint32_t)((2 * m * QS) >> 4), cm = d + (uint32_t)((2 * m * kLaCS) >> 4);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (c < 4 || m < NM)
                                tc_mma_f16_w(taddr + RN * b, cm + (((c >> 2) * kLaCS + 32 * (c & 3)) >> 4),
                                             qm + (((c >> 2) * QS + 32 * (c & 3)) >> 4), IDS, m > 0 || c > 0);
                    }
                    if (!ok) break;
                    tc_commit_w(&bS[b]);
                    ++cs;
                    t.next(KS);
                }
                const int y = x - (KS - 1);
                if (y < 0) continue;
                ok = __all_sync(kFull, mbar_wait_ab(&bP[co & 1], (unsigned)(co >> 1) & 1u, abort));
                if (!ok) break;
                tc_fence_after();
                const uint64_t st = (uint32_t)(u.s * (TB >> 4));
#pragma unroll
                for (int m = 0; m < NM; ++m) {
#pragma unroll
                    for (int c = 0; c < kLatTok / 16; ++c)
                        tc_mma_f16_w(taddr + OC + RN * m, dc + st + ((2 * m * kLaCS + 2048 * c) >> 4),
                                     dp + st + ((2048 * c) >> 4), IDO, y > 0 || c > 0);
                    tc_commit_w(&eC[u.s * NM + m]);
                }
                tc_commit_w(&bF[co & 1]);
                ++co;
                u.next(KS);
            }
            qph ^= 1u;
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        // every MMA and commit has landed before memory is given up (bounded)
        tc_commit_w(bE);
        mbar_wait(bE, 0u);
        __syncwarp();
    } else if (warp == WS + 1) {
        // ---- copies ----
        CkRing t;
        int cnt = 0, parts = 0, meets = 0;   // tiles; parts told of; copies waited for here
        while (ok && walk.next(kg, a, sg)) {
            const int T = sg.T, Tq = a.Tqk[sg.i], n = sg.n;
            const long long new0 = (long long)sg.i * a.n_stride;
            for (int x = 0; x < sg.nx; ++x, ++cnt, t.next(KS)) {
                const LaTile lt(kLatTok * (sg.x0 + x), T, Tq);
                const int kb = lt.tb / kLatTok;
                unsigned char *tile = sC + t.s * TB;
                const unsigned char *ring = (const unsigned char *)(dv.ring + lat_ring(g, sg.i, kb)),
                                    *keys = (const unsigned char *)(dv.kr + lat_kr(g, sg.i, kb));
                // the record after next into L2 (the first two at the start)
                if (lane == 0)
                    for (int e = x ? 2 : 0; e < 3; ++e)
                        if (lt.tb + (e + 1) * kLatTok <= Tq && x + e < sg.nx)
                            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(dv.rec + lat_rec(g, sg.i, kb + e)),
                                         "r"(g.rec_bytes)
                                         : "memory");
                // New tokens: a full tile of them (and of cached ones before them) by
                // TMA; then, over what it brought of the rows before them, the cached
                // ones.  A short one: the cached block, or zeros (what lies behind the
                // last token has no weight, but must be finite), and row by row.
                const int old = min(max(T - lt.tb, 0), kLatTok), rows = T + n - lt.tb;   // cached rows, rows in all
                const bool fresh = !lt.keys, full = rows >= kLatTok;
                if (fresh) {
                    ok = __all_sync(kFull, cnt < KS || mbar_wait_ab(&eC[t.s * NM + NM - 1], t.p ^ 1u, abort));
                    if (!ok) break;
                    if (old > 0 && lane == 0) {
                        mbar_expect_tx(bX, CB + RB);
                        if (full) {
                            for (int c = 0; c < 2 * NM; ++c)
                                tma_sw(tile + c * kLaCS, &tmC, 64 * c, (int)(new0 + lt.tb - T), bX);
                            tma_sw(tile + CB, &tmK, 0, (int)(new0 + lt.tb - T), bX);
                        } else {
                            bulk_g2s(tile, ring, CB, bX);
                            bulk_g2s(tile + CB, keys, RB, bX);
                        }
                    }
                    if (old > 0) {
                        ok = __all_sync(kFull, mbar_wait_ab(bX, (unsigned)meets++ & 1u, abort));
                        if (!ok) break;
                    }
                    if (!full) {
                        constexpr int CR = (RD + kLatRope) / 8;   // 16-byte chunks of a row
                        constexpr int U = 4;
#pragma unroll 1
                        for (int e0 = old * CR + lane; e0 < (old > 0 ? rows : kLatTok) * CR; e0 += 32 * U) {
                            uint4 v[U];
#pragma unroll
                            for (int k = 0; k < U; ++k) {
                                const int e = e0 + 32 * k, r = e / CR, c = e - r * CR;
                                const size_t row = (size_t)(new0 + lt.tb - T + r);
                                v[k] = make_uint4(0u, 0u, 0u, 0u);
                                if (r < rows)
                                    v[k] = *reinterpret_cast<const uint4 *>(c < RD / 8 ? Cn + row * RD + 8 * c
                                                                                       : Kn + row * kLatRope + 8 * (c - RD / 8));
                            }
#pragma unroll
                            for (int k = 0; k < U; ++k) {
                                const int e = e0 + 32 * k, r = e / CR, c = e - r * CR;
                                if (r < kLatTok) *reinterpret_cast<uint4 *>(tile + lat_at(c, r, kLatTok)) = v[k];
                            }
                        }
                        fence_proxy_async();
                        __syncwarp();
                    }
                }
                for (int m = 0; m < NM; ++m, ++parts) {
                    ok = __all_sync(kFull, ok && (cnt < KS || mbar_wait_ab(&eC[t.s * NM + m], t.p ^ 1u, abort)));
                    if (!ok) break;
                    if (lane == 0) {
                        uint64_t *const bar = &bR[t.s * NM + m];
                        unsigned char *dst = tile + 2 * m * kLaCS;
                        if (lt.block) {
                            mbar_expect_tx(bar, 2 * kLaCS);
                            bulk_g2s(dst, ring + 2 * m * kLaCS, 2 * kLaCS, bar);
                        } else if (fresh && full) {
                            mbar_expect_tx(bar, 2 * (old > 0 ? old * 128 : kLaCS));
                            for (int c = 0; c < 2; ++c)
                                if (old > 0) bulk_g2s(dst + c * kLaCS, ring + (2 * m + c) * kLaCS, old * 128, bar);
                                else tma_sw(dst + c * kLaCS, &tmC, 128 * m + 64 * c, (int)(new0 + lt.tb - T), bar);
                        } else {
                            mbar_arrive(bar);
                        }
                    }
                }
                if (!ok) break;
                // (the last part given back: the weights too, O^T's MMAs end in order)
                if (lane == 0) {
                    if (lt.keys || (fresh && full)) {
                        mbar_expect_tx(&bK[t.s], lt.keys || old == 0 ? RB : old * 128);
                        if (lt.keys || old > 0) bulk_g2s(tile + CB, keys, lt.keys ? RB : old * 128, &bK[t.s]);
                        else tma_sw(tile + CB, &tmK, 0, (int)(new0 + lt.tb - T), &bK[t.s]);
                    } else {
                        mbar_arrive(&bK[t.s]);
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            // every copy has landed before shared memory is given up (bounded)
            for (int y = max(0, parts - KS * NM); y < parts; ++y)
                mbar_wait(&bR[y % (KS * NM)], (unsigned)(y / (KS * NM)) & 1u);
            for (int y = max(0, cnt - KS); y < cnt; ++y) mbar_wait(&bK[y % KS], (unsigned)(y / KS) & 1u);
            if (meets > 0) mbar_wait(bX, (unsigned)(meets - 1) & 1u);   // (the one whose wait was given up)
        }
        __syncwarp();
    } else {
        // ---- tiles, softmax, output ----
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const int x0 = warp >> 2, r0 = CN * x0, t0 = 32 * (warp & 3), tok = t0 + lane;   // word, rows, token
        const uint32_t tO = taddr + lane_off + OC + r0, tL = tO + RN * NM;   // O^T, two buffers of each thread's sums
        int cnt = 0, tiles = 0;   // softmax, restored
        CkRing t, u;
        while (walk.next(kg, a, sg)) {
            const int T = sg.T, Tq = a.Tqk[sg.i], nx = sg.nx, first = sg.x0, row0 = sg.row0;
            const unsigned char *rec = dv.rec + lat_rec(g, sg.i, first);
            // Q: row (token, head), 8 rows x 4 chunks at a time; rows past the last
            // are zero (the last segment's scores are all read)
            constexpr int QC = (RD + kLatRope) / 8, QW = kLaWork * 8 / RN, QN = (QC / 4 + QW - 1) / QW;   // chunks of a row; warps and turns of 8 rows
            {
                uint4 v[QN];
                const int q = 8 * (warp / QW) + (lane & 7), c0 = 4 * (warp % QW) + (lane >> 3);
#pragma unroll
                for (int k = 0; k < QN; ++k) {
                    const int c = 4 * QW * k + c0;
                    if (c >= QC) continue;
                    const int rw = min(sg.row0 + q, sg.nrows - 1), tk = chunk_div(a, rw);
                    const size_t row = ((size_t)sg.i * h + rw - tk * h) * a.n_stride + tk;
                    v[k] = *reinterpret_cast<const uint4 *>(c < RD / 8 ? Q + row * RD + 8 * c : Qr + row * kLatRope + 8 * (c - RD / 8));
                }
#pragma unroll
                for (int k = 0; k < QN; ++k) {
                    const int c = 4 * QW * k + c0;
                    if (c >= QC) continue;
                    if (sg.row0 + q >= sg.nrows) v[k] = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(sQ + lat_at(c, q, RN)) = v[k];
                }
            }
            if (tid < RN) s_ref[tid] = kLaUnset;
            if (tid == 0) s_seg = sg;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bQ);
            la_sync();   // the references are set
            const int p0 = T + chunk_div(a, sg.row0);   // the first row's position
            // step x: tile x restored, then the softmax of tile x - (KS - 1)
#pragma unroll 1
            for (int x = 0; x < nx + KS - 1; ++x) {
                // (what follows from the thread's number is formed anew every tile, under names
                // of its own: kept, it would be spilled)
                int th = threadIdx.x;
                asm volatile("" : "+r"(th));
                const int wx = th >> 7, wr = CN * wx, wt = th & 127, w0 = wt & ~31, ln = th & 31;
                const unsigned out = lat_at(wx * (Units::CW / 8), wt, kLatTok);   // unit 0's place in a tile
                if (x < nx) {
                    const LaTile lt(kLatTok * (first + x), T, Tq);
                    unsigned char *tile = sC + t.s * TB;
                    Units cur;   // (from L2; on their way while the parts' places are waited for)
                    if (lt.packed)
                        cur.load(rec + wt * 16 + wx * (kLatTok * 16), rec + g.off_sz + wt * 4, wx * Units::CW, __ffs(g.G) - 1);
                    rec += g.rec_bytes;
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        constexpr int SP = Units::SPAN;
                        if (SP > 1 && wx * Units::CW / 128 != m % SP) continue;   // other warps'
                        if (lt.packed) {
                            // the part's place is free
                            ok = ok && __all_sync(kFull, tiles < KS || mbar_wait_ab(&eC[t.s * NM + m], t.p ^ 1u, abort));
                            if (ok)
#pragma unroll
                                for (int k = Units::PU * (m / SP); k < Units::PU * (m / SP + 1); ++k)
                                    la_restore<BITS>(tile + (Units::WX * k * Units::CW / 64) * kLaCS, out, cur.w[k], cur.sz[k]);
                            fence_proxy_async();
                            __syncwarp();
                        }
                        if (ok && ln == 0) mbar_arrive(&bC[t.s * NM + m]);
                    }
                    ++tiles;
                    t.next(KS);
                }
                const int xs = x - (KS - 1);
                if (xs < 0) continue;
                const int b = cnt & 1, key0 = kLatTok * (first + xs);
                const uint32_t tW = taddr + ((uint32_t)w0 << 16) + wr, wS = tW + RN * b;
                const uint32_t wO = tW + OC, wL = wO + RN * NM;
                // the sums so far, and with this tile (kept apart until the tile stands)
                const uint32_t tL0 = wL + RN * (xs & 1), tL1 = wL + RN * (~xs & 1);
                // rows c < lim do not see this token: those of a token before it
                int lim = 0;
                if (key0 + kLatTok - 1 > p0) {
                    const int l = (key0 + wt - T) * h - row0 - wr;   // (below 2^24 + 2^16)
                    lim = l < 0 ? 0 : l > CN ? CN : l;
                }
                const unsigned sP = smem_u32(sC + u.s * TB + CB) + lat_at(wr / 8, wt, kLatTok);   // (the tile's rotary keys are read once S^T is in)
                ok = ok && __all_sync(kFull, mbar_wait_ab(&bS[b], (unsigned)(cnt >> 1) & 1u, abort));
                tc_fence_after();
                float up = INFINITY;   // (the segment's first tile: a raise at once)
                if (ok && xs > 0) up = la_weights<RN>(wS, tL0, tL1, false, sP, s_ref + wr, sl2, lim);
                if (la_any(!ok || up > kCkLift + kCkLag)) {   // a raise: then this tile's weights anew
                    if (la_any(!ok)) {   // every warp learns whether one has given up
                        ok = false;
                        break;
                    }
                    la_raise<RN>(wS, sl2, lim, s_ref, s_al, s_red);
                    if (xs > 0) {   // O^T, once that of the last tile is in, and the sums
                        ok = __all_sync(kFull, mbar_wait_ab(&bF[~cnt & 1], (unsigned)((cnt - 1) >> 1) & 1u, abort));
                        if (ok) {
                            tc_fence_after();
                            la_rescale<RN, NM>(wO, s_al + wr);
                            la_rescale<RN, 1>(tL0, s_al + wr);
                        }
                    }
                    if (ok) la_weights<RN>(wS, tL0, tL1, xs == 0, sP, s_ref + wr, sl2, lim);
                    if (la_any(!ok)) {
                        ok = false;
                        break;
                    }
                }
                if (th == 0) mbar_arrive(&bP[b]);   // (after the vote: every warp's weights are in)
                ++cnt;
                u.next(KS);
            }
            if (!ok) break;
            ok = __all_sync(kFull, mbar_wait_ab(&bF[~cnt & 1], (unsigned)((cnt - 1) >> 1) & 1u, abort));
            if (la_any(!ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // the rows' sums over the threads: halves exchanged, lane c ends with row c
            float lsum[CN];
            {
                uint32_t l[CN];
                la_ld(tL + RN * (nx & 1), l);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < CN; ++c) lsum[c] = __uint_as_float(l[c]);
            }
#pragma unroll
            for (int o = CN / 2; o; o >>= 1)
#pragma unroll
                for (int c = 0; c < o; ++c) {
                    const bool hi = lane & o;
                    const float give = hi ? lsum[c] : lsum[c + o], keep = hi ? lsum[c + o] : lsum[c];
                    lsum[c] = keep + __shfl_xor_sync(kFull, give, o);
                }
#pragma unroll
            for (int o = CN; o < 32; o <<= 1) lsum[0] += __shfl_xor_sync(kFull, lsum[0], o);
            if (lane < CN) s_red[warp & 3][r0 + lane] = lsum[0];
            la_sync();
            const bool part = nx < s_seg.nt;
            const size_t pr = (size_t)(2 * blockIdx.x + (first == 0 ? 1 : 0)) * RN;
            if (tid < RN) {
                const float l = s_red[0][tid] + s_red[1][tid] + s_red[2][tid] + s_red[3][tid];
                s_al[tid] = 1.f / l;
                if (part && s_seg.row0 + tid < s_seg.nrows)
                    reinterpret_cast<float2 *>(a.ml)[pr + tid] = make_float2(s_ref[tid] == kLaUnset ? -INFINITY : -s_ref[tid], l);
            }
            la_sync();
            // the output: thread = channel, a row at a time; lane c knows where row c
            // begins
            const CkSeg se = s_seg;
            const int rows = min(se.nrows - se.row0 - r0, CN);
            long long off;
            {
                const int q = r0 + lane, rw = min(se.row0 + q, se.nrows - 1), tk = chunk_div(a, rw);
                off = part ? (long long)(pr + q) * RD : (((long long)se.i * h + rw - tk * h) * a.n_stride + tk) * RD;
            }
            const float inv = s_al[r0 + lane];
#pragma unroll 1
            for (int m = 0; m < NM && rows > 0; ++m) {
                uint32_t o[CN];
                la_ld(tO + RN * m, o);
                tc_wait_ld();
                const int ch = 128 * m + tok;
                if (part) {
#pragma unroll
                    for (int c = 0; c < CN; ++c) {
                        const long long at = __shfl_sync(kFull, off, c) + ch;
                        if (c < rows) a.acc[at] = __uint_as_float(o[c]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < CN; ++c) {
                        const long long at = __shfl_sync(kFull, off, c) + ch;
                        const float w = __shfl_sync(kFull, inv, c);
                        if (c < rows) O[at] = __float2half_rn(__uint_as_float(o[c]) * w);
                    }
                }
            }
            tc_fence_before();
            la_sync();   // the sums and references are read
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

// Joins the partials of the row tiles that CTA boundaries cut (a block per
// boundary and RB rows, 8 / RB warps a row that take every so-manieth partial):
// weights 2^(m_k - M), M the largest m.
template <int RD, int RB>
__global__ void __launch_bounds__(256) latent_join_kernel(__half *O, const __grid_constant__ ChunkArgs a) {
    constexpr int W = 8 / RB, V = RD / 128;   // warps a row, 16-byte pieces a lane
    __shared__ __align__(16) float s_acc[RB][W][RD];
    __shared__ float s_l[RB][W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rr = warp / W, w = warp % W;
    const int RN = a.tile_rows, c = blockIdx.x / (RN / RB) + 1, r = blockIdx.x % (RN / RB) * RB + rr;
    const ChunkPos &p = a.cta[c];
    kivi_after_previous<false>();
    if (p.o <= kLaLead) return;   // CTA c starts with a row tile of its own
    const int i = p.i, m = p.m;
    const long long first = p.u - p.o + kLaLead;                         // the unit of its first tile
    if (a.cta[c - 1].u > first) return;                                  // an earlier boundary owns it
    const int nrows = min(a.n[i] * a.hg - m * RN, RN);
    if (blockIdx.x % (RN / RB) * RB >= nrows) return;
    const long long end = first + chunk_tiles(a, i, m);
    int c1 = c;                                                          // the last CTA with its tiles
    while (a.cta[c1 + 1].u < end) ++c1;
    const int c0 = c - 1;   // (holds the first tile, slot 2 c + 1; the others start in it, slot 2 c)
    const float2 *ml = reinterpret_cast<const float2 *>(a.ml);
    float4 acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    if (r < nrows) {
        auto part = [&](int k) { return (size_t)(2 * k + (k == c0 ? 1 : 0)) * RN + r; };
        float M = -INFINITY;
        for (int k = c0 + lane; k <= c1; k += 32) M = fmaxf(M, ml[part(k)].x);
        M = la_redux_max(M);
#pragma unroll 4
        for (int k = c0 + w; k <= c1; k += W) {
            const float2 x = ml[part(k)];
            const float wt = x.x == -INFINITY ? 0.f : ex2(x.x - M);   // (sees nothing of this share)
            const float4 *src = reinterpret_cast<const float4 *>(a.acc + part(k) * RD) + lane;
            L = fmaf(wt, x.y, L);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 y = src[32 * v];
                acc[v].x = fmaf(wt, y.x, acc[v].x);
                acc[v].y = fmaf(wt, y.y, acc[v].y);
                acc[v].z = fmaf(wt, y.z, acc[v].z);
                acc[v].w = fmaf(wt, y.w, acc[v].w);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) reinterpret_cast<float4 *>(s_acc[rr][w])[lane + 32 * v] = acc[v];
    if (lane == 0) s_l[rr][w] = L;
    __syncthreads();
    if (r >= nrows) return;
    // the row's warps share its channels, two a thread and turn
    float l = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) l += s_l[rr][k];
    const float inv = 1.f / l;
    const int row = m * RN + r, tok = chunk_div(a, row);
    __half *dst = O + (((size_t)i * a.hq + row - tok * a.hg) * a.n_stride + tok) * RD;
    for (int e = 2 * (32 * w + lane); e < RD; e += 64 * W) {
        float2 y = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float2 z = *reinterpret_cast<const float2 *>(&s_acc[rr][k][e]);
            y.x += z.x;
            y.y += z.y;
        }
        *reinterpret_cast<uint32_t *>(dst + e) = ck_pack(y.x * inv, y.y * inv);
    }
}

template <int RD, int BITS, int RN>
cudaError_t launch(const LatentGeom &g, const LatentDev &dv, const __half *Q, const __half *Qr, const __half *C,
                   const __half *Kr, __half *O, const ChunkArgs &a, const ChunkPlan &plan, float scale, int device,
                   cudaStream_t st) {
    static std::atomic<uint64_t> done;
    CUtensorMap tc, tk;
    const long long rows = (long long)g.b * a.n_stride;
    cudaError_t e = make_sw_map(&tc, C, rows, RD, kLatTok);
    if (e == cudaSuccess) e = make_sw_map(&tk, Kr, rows, kLatRope, kLatTok);
    if (e == cudaSuccess) e = kivi_allow_smem(latent_attn_kernel<RD, BITS, RN>, la_smem(RD, RN), device, done);
    if (e != cudaSuccess) return e;
    e = kivi_launch_after(latent_attn_kernel<RD, BITS, RN>, dim3((unsigned)plan.ctas), kLaThreads, la_smem(RD, RN), st, 1, g, dv, Q, Qr, C,
                          Kr, O, tc, tk, scale * 1.4426950408889634f, a);
    if (e != cudaSuccess || !plan.join) return e;
    long long tiles = 0;
    for (int i = 0; i < g.b; ++i) tiles += chunk_row_tiles(a, i);
    // many partials a row tile: all of a block's warps at one row
    const bool one = plan.ctas > 8 * tiles;
    return kivi_launch_after(one ? latent_join_kernel<RD, 1> : latent_join_kernel<RD, 4>,
                             dim3((unsigned)((plan.ctas - 1) * (one ? RN : RN / 4))), 256, 0, st, 1, O, a);
}

}  // namespace

bool kivi_plan_latent(const LatentGeom &g, int h, ChunkArgs &a, int num_sms, ChunkPlan *plan) {
    a.hq = a.hg = h;
    a.hg_mul = (unsigned)(((1ull << 32) + h - 1) / h);
    a.vis = Visible{0, 0};
    a.tile_blocks = kLatTok / KIVI_KBLK;
    // Row tiles of 32 where they are hardly more: a tile then takes 0.7 to 0.9 of the time
    // (8 x 16k 4-bit tokens: 32 rows a sequence 43.6 us for 49.9 with r = 512, 24.5 for
    // 28.2 with 256; 96 rows, three tiles for two, 98 for 87 and 49 for 44).
    long long few = 0, many = 0;   // tiles
    for (int i = 0; i < g.b; ++i) {
        const long long rows = (long long)a.n[i] * h, tiles = (a.T[i] + a.n[i] + kLatTok - 1) / kLatTok;
        few += (rows + kLatFew - 1) / kLatFew * tiles;
        many += (rows + kLatRows - 1) / kLatRows * tiles;
    }
    a.tile_rows = 3 * few < 4 * many ? kLatFew : kLatRows;
    *plan = ChunkPlan{false, false, 0};
    // (shares of two units and more: a tile takes as long as 8 of the chunk attention's)
    return kivi_plan_units(g.b, 1, a, num_sms, kLaLead, 2, &plan->ctas, &plan->join);
}

size_t kivi_latent_partial_floats(const LatentGeom &g, int num_sms) {
    return (size_t)2 * num_sms * kLatRows * (g.r + 2);
}

cudaError_t kivi_launch_latent_attn(const LatentGeom &g, const LatentDev &dv, const __half *Q, const __half *Qr,
                                    const __half *C, const __half *Kr, __half *O, ChunkArgs &a, const ChunkPlan &plan,
                                    float scale, float *partials, int device, int num_sms, cudaStream_t st) {
    a.acc = partials;
    a.ml = partials + (size_t)2 * num_sms * kLatRows * g.r;
    const auto pick = [&](auto rd, auto bits) {
        return a.tile_rows == kLatRows
                   ? launch<rd(), bits(), kLatRows>(g, dv, Q, Qr, C, Kr, O, a, plan, scale, device, st)
                   : launch<rd(), bits(), kLatFew>(g, dv, Q, Qr, C, Kr, O, a, plan, scale, device, st);
    };
    using I2 = std::integral_constant<int, 2>;
    using I4 = std::integral_constant<int, 4>;
    using I256 = std::integral_constant<int, 256>;
    using I512 = std::integral_constant<int, 512>;
    if (g.r == 256) return g.bits == 2 ? pick(I256(), I2()) : pick(I256(), I4());
    return g.bits == 2 ? pick(I512(), I2()) : pick(I512(), I4());
}
