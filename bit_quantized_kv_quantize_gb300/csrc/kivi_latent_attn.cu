// kivi_latent_attn.cu -- latent attention in its absorbed form: new tokens over
// the quantized latent cache and over themselves, on the 5th-generation tensor
// cores.
//
// Mathematics.  With q = [Wk_h^T qn ; qr] (r + 64 channels) and a token's
// row t_s = [c_s ; kr_s], head h of the token at position p has
//   out = sum_s softmax_s(scale q . t_s) c_s   over s <= p:
// one key and value row a token for every head.  So the rows (token, head) of a
// sequence are one list, cut into row tiles of 64, and a tile of 64 tokens,
// restored once to fp16 in shared memory, is the B operand of
//   S [64 rows x 64 tokens] = Q T^T   (r + 64 deep)
// and, read along its other axis, the A operand of
//   O^T [r x 64 rows] += C^T P^T      (64 deep, r / 128 MMAs of 128 rows).
// O is held transposed because 128 channels fill the tensor memory's lanes
// where 64 rows would fill half of them: r x 64 sums take r / 2 columns.
//
// The softmax has one row in the four threads of a quad (each holds 16 of its
// 64 scores), weights against a lifted reference as in the chunk attention;
// the reference is raised, and O^T's columns rescaled, only when a score lies
// more than 2^8 above it.
//
// Rounding.  A restored latent vector (scale code + zero), the weights and the
// query enter the products in fp16 (2^-11 relative each); sums in fp32.
//
// Work split (as the chunk attention's): the 64-token tiles of all row tiles
// end to end, each CTA an equal share, cut row tiles joined from partials.
#include <cstring>

#include "kivi_chunk_tiles.cuh"
#include "kivi_latent.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_tma.cuh"

namespace {

constexpr int kLaDq = 8;   // warps that restore tiles
constexpr int kLaThreads = 32 * (4 + kLaDq + 3);
constexpr unsigned kLaCS = KIVI_KBLK * 16;   // bytes from a 16-byte chunk of a tile to the next along its rows
__host__ __device__ constexpr int la_stages(int r) { return r == 512 ? 2 : 4; }
__host__ __device__ constexpr int la_tile(int r) { return (r + kLatRope) / 8 * (int)kLaCS; }   // bytes: of Q too
__host__ __device__ constexpr size_t la_smem(int r) { return (size_t)(la_stages(r) + 1) * la_tile(r) + kLatRows * KIVI_KBLK * 2; }

// whether any of the four softmax warps says v (all come here every tile)
__device__ __forceinline__ bool la_any(bool v) {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void la_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

// 16 bytes of codes of a token (word x) to 128 / BITS channels of it: sz the
// scales and zeros of the groups they span (GW channels of the word each).
template <int BITS, int NG>
__device__ __forceinline__ void la_restore(unsigned char *dst, const uint4 &v, const uint32_t (&sz)[NG]) {
    constexpr int PW = 32 / BITS, CW = 4 * PW;   // channels a 32-bit word, the 16 bytes
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
        *reinterpret_cast<uint4 *>(dst + c * kLaCS) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// A warp's part of a fully quantized tile in registers: its units are half a
// block's tokens (a lane each) of one 16-byte word.
template <int RD, int BITS, int GL>   // GL: log2 of the group size
struct LaPacked {
    static constexpr int CW = 128 / BITS, NU = 2 * RD / CW / kLaDq;   // channels a word, units a warp
    static constexpr int NG = CW >> GL > 1 ? CW >> GL : 1;            // groups a word spans
    uint4 w[NU];
    uint32_t sz[NU][NG];
    __device__ __forceinline__ void load(const unsigned char *rec, int off_sz, int warp, int lane) {
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int u = warp + kLaDq * k, x = u >> 1, t = 32 * (u & 1) + lane;
            w[k] = __ldg(reinterpret_cast<const uint4 *>(rec + (x * KIVI_KBLK + t) * 16));
#pragma unroll
            for (int q = 0; q < NG; ++q)
                sz[k][q] = __ldg(reinterpret_cast<const uint32_t *>(rec + off_sz + ((((x * CW) >> GL) + q) * KIVI_KBLK + t) * 4));
        }
    }
    __device__ __forceinline__ void restore(unsigned char *tile, int warp, int lane) const {
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int u = warp + kLaDq * k, x = u >> 1, t = 32 * (u & 1) + lane;
            la_restore<BITS, NG>(tile + x * (CW / 8) * kLaCS + t * 16, w[k], sz[k]);
        }
    }
};

// 16 bytes (8 channels, chunk c) of token tau's row: from the codes, the ring or
// the new tokens; zero past them.
__device__ __forceinline__ uint4 la_row16(const LatentGeom &g, const LatentDev &dv, const __half *Cn, const __half *Kn,
                                          int i, int T, int Tq, int n, size_t new0, int tau, int c) {
    const int kb = tau / KIVI_KBLK, t = tau % KIVI_KBLK, nc = g.r / 8;
    if (tau >= T + n) return make_uint4(0u, 0u, 0u, 0u);
    if (tau >= T)
        return *reinterpret_cast<const uint4 *>(c < nc ? Cn + (new0 + (tau - T)) * g.r + 8 * c
                                                       : Kn + (new0 + (tau - T)) * kLatRope + 8 * (c - nc));
    if (c >= nc) return *reinterpret_cast<const uint4 *>(dv.kr + lat_kr(g, i, kb) + ((c - nc) * KIVI_KBLK + t) * 8);
    if (tau >= Tq) return *reinterpret_cast<const uint4 *>(dv.ring + lat_ring(g, i, kb) + ((size_t)c * KIVI_KBLK + t) * 8);
    const unsigned char *rec = dv.rec + lat_rec(g, i, kb);
    const __half2 sz = *reinterpret_cast<const __half2 *>(rec + g.off_sz + ((8 * c / g.G) * KIVI_KBLK + t) * 4);
    const int PW = 32 / g.bits, wi = 8 * c / PW, f0 = (8 * c % PW) >> 1, m = (1 << g.bits) - 1;
    const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + ((wi >> 2) * KIVI_KBLK + t) * 16 + (wi & 3) * 4);
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int lo = (w >> (g.bits * (f0 + k))) & m, hi = (w >> (16 + g.bits * (f0 + k))) & m;
        h[k] = h2u(__hfma2(__halves2half2(__int2half_rn(lo), __int2half_rn(hi)), __low2half2(sz), __high2half2(sz)));
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// What a tile holds, and who fills it.
struct LaTile {
    int tb;
    bool packed;   // codes only
    bool ring;     // a whole block of the ring: copied
    bool fresh;    // new tokens only: copied
    bool keys;     // the rotary keys are a whole block of the cache: copied
    __device__ __forceinline__ LaTile(int tb, int T, int Tq, int n)
        : tb(tb), packed(tb + KIVI_KBLK <= Tq), ring(tb >= Tq && tb + KIVI_KBLK <= T),
          fresh(tb >= T && tb + KIVI_KBLK <= T + n), keys(tb + KIVI_KBLK <= T) {}
};

// A tile that is neither: chunk by chunk, by all restoring warps.
__device__ __noinline__ void la_mixed(const LatentGeom &g, const LatentDev &dv, const __half *Cn, const __half *Kn,
                                      unsigned char *tile, const LaTile &lt, int i, int T, int Tq, int n, size_t new0) {
    constexpr int U = 4;
    const int e0 = threadIdx.x - 128;   // (the restoring warps follow the four of the softmax)
    const int total = (lt.keys ? g.r / 8 : (g.r + kLatRope) / 8) * KIVI_KBLK;
    for (int e = e0; e < total; e += U * 32 * kLaDq) {
        uint4 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int y = min(e + k * 32 * kLaDq, total - 1);
            x[k] = la_row16(g, dv, Cn, Kn, i, T, Tq, n, new0, lt.tb + y % KIVI_KBLK, y / KIVI_KBLK);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int y = e + k * 32 * kLaDq;
            if (y < total) *reinterpret_cast<uint4 *>(tile + y * 16) = x[k];
        }
    }
}

// One restoring warp's share of a segment's nx tiles from first token tb0 on.
// False if a wait ran out.
template <int RD, int BITS, int GL>
__device__ __forceinline__ bool la_tiles(const LatentGeom &g, const LatentDev &dv, const __half *Cn, const __half *Kn,
                                         int i, int T, int Tq, int n, size_t new0, int tb0, int nx, int &tiles, CkRing &t,
                                         unsigned char *sC, uint64_t *bC, uint64_t *eC, const volatile int *abort) {
    constexpr int KS = la_stages(RD), TB = la_tile(RD);
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 4;
    LaPacked<RD, BITS, GL> cur, nxt;
    const unsigned char *rec = dv.rec + lat_rec(g, i, tb0 / KIVI_KBLK);
    if (tb0 + KIVI_KBLK <= Tq) cur.load(rec, g.off_sz, warp, lane);
#pragma unroll 1
    for (int x = 0; x < nx; ++x, ++tiles, t.next(KS)) {
        const LaTile lt(tb0 + KIVI_KBLK * x, T, Tq, n);
        unsigned char *tile = sC + t.s * TB;
        if (lt.packed && lt.tb + 2 * KIVI_KBLK <= Tq && x + 1 < nx)
            nxt.load(rec + (size_t)(x + 1) * g.rec_bytes, g.off_sz, warp, lane);
        const bool ok = tiles < KS || mbar_wait_ab(&eC[t.s], t.p ^ 1u, abort);
        if (!__all_sync(kFull, ok)) return false;
        if (lt.packed) {
            cur.restore(tile, warp, lane);
            cur = nxt;
        } else if (!lt.ring && !lt.fresh) {
            la_mixed(g, dv, Cn, Kn, tile, lt, i, T, Tq, n, new0);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bC[t.s]);
    }
    return true;
}

// Warps 0-3: softmax and output; 4-11: restoring tiles; 12: S; 13: O^T; 14:
// copies (rotary keys, whole fp16 tiles).  They meet on mbarriers only (bounded
// waits).  Tensor memory: two S buffers of 64 columns, then O^T.  Shared
// memory: tiles [r + 64 channels in chunks of 8][64 tokens], Q alike, P.
template <int RD>
__global__ void __launch_bounds__(kLaThreads, 1)
    latent_attn_kernel(const __grid_constant__ LatentGeom g, const __grid_constant__ LatentDev dv, const __half *__restrict__ Q, const __half *__restrict__ Qr,
                       const __half *__restrict__ Cn, const __half *__restrict__ Kn, __half *__restrict__ O,
                       const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmK, float sl2,
                       const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int KS = la_stages(RD), TB = la_tile(RD), NM = RD / 128;
    constexpr int OC = 2 * KIVI_KBLK;   // first column of O^T
    unsigned char *sC = smem, *sQ = sC + KS * TB, *sP = sQ + TB;
    // counts 4 (the softmax warps): Q, P [buffer of S]; 8: tiles restored; 1: the others
    constexpr int NB = 3 + 3 * KS + 3;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bQ = bars, *const bP = bars + 1, *const bC = bars + 3, *const bB = bC + KS, *const eC = bB + KS,
                    *const bS = eC + KS, *const bF = bS + 2;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;
    __shared__ __align__(16) float s_al[kLatRows];   // a raise's factors; 1 / sum of each row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = a.hg;
    if (tid < NB) {
        mbar_init(&bars[tid], tid < 3 ? 4 : tid < 3 + KS ? kLaDq : 1);
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
    KiviGeom kg;   // (the walk reads b and h)
    kg.b = g.b;
    kg.h = 1;
    CkWalk walk;
    walk.start(a, blockIdx.x);
    CkSeg sg = {};
    constexpr int WS = 4 + kLaDq;

    if (warp == WS) {
        // ---- S = Q T^T ----
        constexpr uint32_t ID = tc_idesc_f16(kLatRows, KIVI_KBLK, 0);
        CkRing t;
        int cnt = 0;
        unsigned qph = 0;
        const uint64_t dq = tc_desc(sQ, kLaCS, 128), dc = tc_desc(sC, kLaCS, 128);
        while (ok && walk.next(kg, a, sg)) {
            const int nx = __reduce_max_sync(kFull, sg.nx);
            for (int x = 0; x < nx; ++x, ++cnt, t.next(KS)) {
                const int b = cnt & 1;
                // Q and the tile in, the buffer's last scores read (their weights written)
                ok = (x > 0 || mbar_wait_ab(bQ, qph, abort)) && mbar_wait_ab(&bB[t.s], t.p, abort) &&
                     mbar_wait_ab(&bC[t.s], t.p, abort) &&
                     (cnt < 2 || mbar_wait_ab(&bP[b], (unsigned)((cnt >> 1) + 1) & 1u, abort));
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t d = dc + (uint32_t)(t.s * (TB >> 4));
#pragma unroll 4
                for (int c = 0; c < (RD + kLatRope) / 16; ++c)
                    tc_mma_f16_w(taddr + KIVI_KBLK * b, dq + ((2 * c * kLaCS) >> 4), d + ((2 * c * kLaCS) >> 4), ID, c > 0);
                tc_commit_w(&bS[b]);
            }
            qph ^= 1u;
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        // every commit has landed before shared memory is given up (bounded)
        for (int y = max(0, cnt - 2); y < cnt; ++y) mbar_wait(&bS[y & 1], (unsigned)(y >> 1) & 1u);
        __syncwarp();
    } else if (warp == WS + 1) {
        // ---- O^T += C^T P^T ----
        constexpr uint32_t ID = tc_idesc_f16_at(128, kLatRows);
        CkRing t;
        int cnt = 0;
        const uint64_t dc = tc_desc(sC, 128, kLaCS), dp = tc_desc(sP, kLaCS, 128);
        while (ok && walk.next(kg, a, sg)) {
            const int nx = __reduce_max_sync(kFull, sg.nx);
            for (int x = 0; x < nx; ++x, ++cnt, t.next(KS)) {
                ok = __all_sync(kFull, mbar_wait_ab(&bP[cnt & 1], (unsigned)(cnt >> 1) & 1u, abort));
                if (!ok) break;
                tc_fence_after();
                const uint64_t d = dc + (uint32_t)(t.s * (TB >> 4));
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int c = 0; c < KIVI_KBLK / 16; ++c)
                        tc_mma_f16_w(taddr + OC + kLatRows * m, d + ((16 * m * kLaCS + 256 * c) >> 4),
                                     dp + ((2 * c * kLaCS) >> 4), ID, x > 0 || c > 0);
                tc_commit_w(bF);
                tc_commit_w(&eC[t.s]);
            }
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        if (cnt > 0) mbar_wait(bF, (unsigned)(cnt - 1) & 1u);
        for (int y = max(0, cnt - KS); y < cnt; ++y) mbar_wait(&eC[y % KS], (unsigned)(y / KS) & 1u);
        __syncwarp();
    } else if (warp == WS + 2) {
        // ---- copies (lane 0 issues) ----
        CkRing t;
        int cnt = 0;
        while (ok && walk.next(kg, a, sg)) {
            if (lane == 0) {
                const int T = sg.T, Tq = a.Tqk[sg.i];
                for (int x = 0; x < sg.nx; ++x, ++cnt, t.next(KS)) {
                    ok = cnt < KS || mbar_wait_ab(&eC[t.s], t.p ^ 1u, abort);
                    if (!ok) break;
                    const LaTile lt(sg.key0(x), T, Tq, sg.n);
                    unsigned char *tile = sC + t.s * TB;
                    constexpr unsigned CB = RD / 8 * kLaCS, RB = kLatRope / 8 * kLaCS;
                    const int kb = lt.tb / KIVI_KBLK;
                    const unsigned bytes = (lt.ring || lt.fresh ? CB : 0u) + (lt.keys || lt.fresh ? RB : 0u);
                    if (bytes) mbar_expect_tx(&bB[t.s], bytes);
                    else mbar_arrive(&bB[t.s]);
                    if (lt.fresh) {
                        const int row = (int)((size_t)sg.i * a.n_stride + (lt.tb - T));
                        tma_box(tile, &tmC, row, &bB[t.s]);
                        tma_box(tile + CB, &tmK, row, &bB[t.s]);
                    } else {
                        if (lt.ring) bulk_g2s(tile, dv.ring + lat_ring(g, sg.i, kb), CB, &bB[t.s]);
                        if (lt.keys) bulk_g2s(tile + CB, dv.kr + lat_kr(g, sg.i, kb), RB, &bB[t.s]);
                    }
                }
            }
            ok = __all_sync(kFull, ok);
        }
        if (lane == 0) {
            if (!ok) {
                s_abort = 1;
                atomicOr(dv.status, KIVI_FLAG_WAIT);
            }
            // every copy has landed before shared memory is given up (bounded)
            for (int y = max(0, cnt - KS); y < cnt; ++y) mbar_wait(&bB[y % KS], (unsigned)(y / KS) & 1u);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---- tiles ----
        int tiles = 0;
        CkRing t;
        while (ok && walk.next(kg, a, sg)) {
            const int T = sg.T, Tq = a.Tqk[sg.i], n = sg.n, tb0 = sg.key0(0), nx = sg.nx;
            const size_t new0 = (size_t)sg.i * a.n_stride;
#define LA_TILES(B, L) la_tiles<RD, B, L>(g, dv, Cn, Kn, sg.i, T, Tq, n, new0, tb0, nx, tiles, t, sC, bC, eC, abort)
            if (g.bits == 4)
                ok = g.G == 32 ? LA_TILES(4, 5) : g.G == 64 ? LA_TILES(4, 6) : LA_TILES(4, 7);
            else
                ok = g.G == 32 ? LA_TILES(2, 5) : g.G == 64 ? LA_TILES(2, 6) : LA_TILES(2, 7);
#undef LA_TILES
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(dv.status, KIVI_FLAG_WAIT);
        }
        __syncwarp();
    } else {
        // ---- softmax ----
        const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
        const int rq = 16 * warp + (lane >> 2), tq = lane & 3;   // this quad's rows: rq, rq + 8
        int cnt = 0;
        while (walk.next(kg, a, sg)) {
            // Q: row (token, head); rows past the last are zero (the last
            // segment's scores are all read)
            for (int e = tid; e < kLatRows * (RD + kLatRope) / 8; e += 128) {
                const int c = e / (2 * kLatRows) * 2 + (e & 1), q = (e >> 1) % kLatRows, rw = sg.row0 + q;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (rw < sg.nrows) {
                    const int tok = chunk_div(a, rw);
                    const size_t row = ((size_t)sg.i * h + rw - tok * h) * a.n_stride + tok;
                    v = *reinterpret_cast<const uint4 *>(c < RD / 8 ? Q + row * RD + 8 * c : Qr + row * kLatRope + 8 * (c - RD / 8));
                }
                *reinterpret_cast<uint4 *>(sQ + c * kLaCS + q * 16) = v;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bQ);
            const int p0 = sg.T + chunk_div(a, sg.row0);   // the first row's position
            const int pos[2] = {sg.T + chunk_div(a, sg.row0 + rq), sg.T + chunk_div(a, sg.row0 + rq + 8)};
            float ref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
            for (int x = 0; x < sg.nx; ++x, ++cnt) {
                const int b = cnt & 1, key0 = sg.key0(x);
                ok = ok && __all_sync(kFull, mbar_wait_ab(&bS[b], (unsigned)(cnt >> 1) & 1u, abort));
                tc_fence_after();
                uint32_t r[32];   // r[4 k + 2 e + c]: row rq + 8 e, token 8 k + 2 tq + c
                float alpha[2] = {1.f, 1.f};
                bool grow = false;
                if (ok) {
                    tc_ld_16x64(taddr + lane_off + KIVI_KBLK * b, r);
                    tc_wait_ld();
                    if (key0 + KIVI_KBLK - 1 > p0) {   // some row does not see the whole tile
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (key0 + 8 * (k >> 2) + 2 * tq + (k & 1) > pos[(k >> 1) & 1]) r[k] = 0xff800000u;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = __uint_as_float(r[2 * e]);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            m = fmaxf(m, fmaxf(__uint_as_float(r[4 * k + 2 * e]), __uint_as_float(r[4 * k + 2 * e + 1])));
                        m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
                        m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
                        if (m != -INFINITY && (ref[e] == -INFINITY || fmaf(m, sl2, -ref[e]) > kCkLift + kCkLag)) {
                            const float up = fmaf(m, sl2, -kCkLift);
                            if (ref[e] != -INFINITY) {
                                alpha[e] = ex2(ref[e] - up);
                                grow = true;
                            }
                            ref[e] = up;
                        }
                    }
                }
                const bool raise = la_any(!ok || grow);
                if (raise && la_any(!ok)) {   // every warp learns whether one has given up
                    ok = false;
                    break;
                }
                uint32_t pw[16];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ms = ref[e] == -INFINITY ? 0.f : ref[e];   // (nothing seen yet: weights 0)
                    float l = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float y0 = ex2(fmaf(__uint_as_float(r[4 * k + 2 * e]), sl2, -ms)),
                                    y1 = ex2(fmaf(__uint_as_float(r[4 * k + 2 * e + 1]), sl2, -ms));
                        l += y0 + y1;
                        pw[2 * k + e] = ck_pack(y0, y1);
                    }
                    lsum[e] = lsum[e] * alpha[e] + l;
                }
                // the last tile's O^T is in: its weights are read, and it may be rescaled
                if (x > 0) ok = __all_sync(kFull, mbar_wait_ab(bF, (unsigned)(cnt - 1) & 1u, abort));
                if (raise) {
                    if (la_any(!ok)) {
                        ok = false;
                        break;
                    }
                    if (tq == 0) {
                        s_al[rq] = alpha[0];
                        s_al[rq + 8] = alpha[1];
                    }
                    la_sync();
                    if (x > 0) {
                        tc_fence_after();
#pragma unroll 1
                        for (int m = 0; m < 2 * NM; ++m) {
                            const uint32_t tO = taddr + lane_off + OC + 32 * m;
                            uint32_t o[32];
                            tc_ld32(tO, o);
                            tc_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                o[c] = __float_as_uint(__uint_as_float(o[c]) * s_al[(32 * m & 32) + c]);
                            tc_st32(tO, o);
                        }
                        tc_wait_st();
                    }
                    la_sync();   // the factors are read
                }
                if (!ok) continue;   // the next vote ends it for every warp
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    *reinterpret_cast<uint32_t *>(sP + k * kLaCS + rq * 16 + tq * 4) = pw[2 * k];
                    *reinterpret_cast<uint32_t *>(sP + k * kLaCS + (rq + 8) * 16 + tq * 4) = pw[2 * k + 1];
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bP[b]);
            }
            ok = ok && __all_sync(kFull, mbar_wait_ab(bF, (unsigned)(cnt - 1) & 1u, abort));
            if (la_any(!ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // the rows' sums, and the output: thread = channel, a row at a time
            const bool part = sg.nx < sg.nt;
            const size_t pr = (size_t)(2 * blockIdx.x + (sg.x0 == 0 ? 1 : 0)) * kLatRows;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                lsum[e] += __shfl_xor_sync(kFull, lsum[e], 1);
                lsum[e] += __shfl_xor_sync(kFull, lsum[e], 2);
                if (tq == 0) {
                    s_al[rq + 8 * e] = 1.f / lsum[e];
                    if (part && sg.row0 + rq + 8 * e < sg.nrows)
                        reinterpret_cast<float2 *>(a.ml)[pr + rq + 8 * e] = make_float2(ref[e], lsum[e]);
                }
            }
            la_sync();
            const int rows = min(sg.nrows - sg.row0, kLatRows), chan = 32 * warp + lane;
#pragma unroll 1
            for (int m = 0; m < 2 * NM; ++m) {
                const int q0 = 32 * (m & 1);
                if (q0 >= rows) continue;
                uint32_t o[32];
                tc_ld32(taddr + lane_off + OC + 32 * m, o);
                tc_wait_ld();
                const int ch = 128 * (m >> 1) + chan;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const int q = q0 + c;
                    if (q >= rows) break;
                    if (part) {
                        a.acc[(pr + q) * RD + ch] = __uint_as_float(o[c]);
                    } else {
                        const int rw = sg.row0 + q, tok = chunk_div(a, rw);
                        O[(((size_t)sg.i * h + rw - tok * h) * a.n_stride + tok) * RD + ch] =
                            __float2half_rn(__uint_as_float(o[c]) * s_al[q]);
                    }
                }
            }
            tc_fence_before();
            la_sync();   // the factors are read
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

template <int RD>
cudaError_t launch(const LatentGeom &g, const LatentDev &dv, const __half *Q, const __half *Qr, const __half *C,
                   const __half *Kr, __half *O, const ChunkArgs &a, const ChunkPlan &plan, float scale, cudaStream_t st) {
    CUtensorMap tc, tk;
    const long long rows = (long long)g.b * a.n_stride;
    cudaError_t e = make_tile_map(&tc, C, rows, RD, KIVI_KBLK);
    if (e == cudaSuccess) e = make_tile_map(&tk, Kr, rows, kLatRope, KIVI_KBLK);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(latent_attn_kernel<RD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)la_smem(RD));
    if (e != cudaSuccess) return e;
    latent_attn_kernel<RD><<<plan.ctas, kLaThreads, la_smem(RD), st>>>(g, dv, Q, Qr, C, Kr, O, tc, tk,
                                                                      scale * 1.4426950408889634f, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || !plan.join) return e;
    const unsigned blocks = (unsigned)(plan.ctas - 1) * (kLatRows / kJoinRows);
    chunk_join_kernel<RD><<<blocks, 256, 0, st>>>(O, a);
    return cudaGetLastError();
}

}  // namespace

bool kivi_plan_latent(const LatentGeom &g, int h, ChunkArgs &a, int num_sms, ChunkPlan *plan) {
    a.hq = a.hg = h;
    a.hg_mul = (unsigned)(((1ull << 32) + h - 1) / h);
    a.vis = Visible{0, 0};
    a.tile_rows = kLatRows;
    a.tile_blocks = 1;
    *plan = ChunkPlan{false, false, 0};
    return kivi_plan_units(g.b, 1, a, num_sms, 2 * kCkLead, &plan->ctas, &plan->join);
}

size_t kivi_latent_partial_floats(const LatentGeom &g, int num_sms) {
    return (size_t)2 * num_sms * kLatRows * (g.r + 2);
}

cudaError_t kivi_launch_latent_attn(const LatentGeom &g, const LatentDev &dv, const __half *Q, const __half *Qr,
                                    const __half *C, const __half *Kr, __half *O, ChunkArgs &a, const ChunkPlan &plan,
                                    float scale, float *partials, int num_sms, cudaStream_t st) {
    a.acc = partials;
    a.ml = partials + (size_t)2 * num_sms * kLatRows * g.r;
    return g.r == 256 ? launch<256>(g, dv, Q, Qr, C, Kr, O, a, plan, scale, st)
                      : launch<512>(g, dv, Q, Qr, C, Kr, O, a, plan, scale, st);
}
