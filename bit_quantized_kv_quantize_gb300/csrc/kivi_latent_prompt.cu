// kivi_latent_prompt.cu -- latent attention in its expanded form: the causal
// attention of a prompt, or of a long chunk behind cached tokens, whose heads' keys
// and values have been formed, on the 5th-generation tensor cores, and the entry
// points kivi_latent_prompt_attn and kivi_latent_expanded_attn.
//
// Mathematics.  Token s of head e has the key [k_s ; kr_s] (128 channels of its
// own, 64 rotary ones that all heads share) and the value v_s [128]:
//   out_p = sum_{s <= p} softmax_s(scale (qn_p . k_s + qr_p . kr_s)) v_s.
// 640 operations a (row, token) where the absorbed form takes 2 (2 r + 64):
// 3.4 times fewer at r = 512, which pays for forming the keys and values as soon
// as more than a few hundred rows share them.
//
// A CTA takes 256 rows (two slots of 128) of one head and walks the 64-token
// tiles up to its last row; S = Q K^T is 192 deep, the rotary keys' tile beside
// the head's in shared memory.  S, the weights and O stay in tensor memory, a
// thread a row; the two slots' softmax and products overlap.  Blocks with the
// most tiles are launched first.
//
// Few row tiles over many tokens would leave SMs idle: then the CTAs of a cluster, up
// to 8, share a row tile's key tiles.  Each leaves its rows' sums and references in
// its shared memory, and joins a part of the rows from all of them there (no
// workspace, no second kernel, the same order always).  1024 tokens of 16 heads over
// 8000: the whole call 126 us for 177; 256 over 30,000: 269 for 591.
#include <cooperative_groups.h>

#include <climits>
#include <cstring>

#include "../../include/kivi.h"
#include "kivi_chunk_tiles.cuh"
#include "kivi_latent.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_tma.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kLpMaxSplit = 8;   // CTAs that share a row tile
constexpr int kLpJoin = 4;       // key tiles that take as long as a join
constexpr int kLpRows = 128, kLpKeys = KIVI_KBLK, kLpStages = 3;
constexpr int kLpQK = kLatHead + kLatRope;
constexpr int kLpThreads = 32 * 12;
constexpr int kLpQ = kLpRows * kLpQK * 2, kLpK = kLpKeys * kLpQK * 2, kLpV = kLpKeys * kLatHead * 2;
constexpr size_t kLpSmem = (size_t)2 * kLpQ + (size_t)kLpStages * (kLpK + kLpV) + 1024;
constexpr int kLpQs = kLpRows * 128, kLpKs = kLpKeys * 128;   // a tile of 64 channels (bytes)

struct PromptArgs {
    __half *out;
    int b, h, n_stride, s_stride, mt;   // strides of queries and of keys; row tiles of the longest sequence
    int split;                          // CTAs (a cluster) that share a row tile's key tiles
    float sl2;                          // scale log2(e)
    unsigned *status;
    int n[KIVI_MAX_BATCH], T[KIVI_MAX_BATCH];   // queries of a sequence; tokens before them
};

__device__ __forceinline__ unsigned long long lp_f2(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void lp_f2(unsigned long long v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long lp_fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long lp_add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Warps 0-7: softmax and output (thread tid owns row tid mod 128 of slot tid /
// 128; tensor-memory columns [256 slot, + 256): S in 0-63, weights from 64 and
// 96, O from 128); 8, 9: S of a slot; 10: O += P V; 11: copies.
__global__ void __launch_bounds__(kLpThreads, 1)
    latent_prompt_kernel(const __grid_constant__ CUtensorMap tmQn, const __grid_constant__ CUtensorMap tmQr,
                         const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmKr,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PromptArgs a) {
    extern __shared__ unsigned char raw[];
    unsigned char *const smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    constexpr int KS = kLpStages;
    const int bh = a.b * a.h, blk = blockIdx.x / a.split, rank = blockIdx.x % a.split;
    const int pair = blk % bh, m = a.mt - 1 - blk / bh, i = pair / a.h;
    const int n = a.n[i], T = a.T[i], row0 = m * 2 * kLpRows;
    if (row0 >= n) {
        kivi_after_previous();
        return;
    }
    unsigned char *sQ = smem, *sK = sQ + 2 * kLpQ, *sV = sK + KS * kLpK;
    // counts 4 (a slot's softmax warps): P [slot][buffer], scores read [slot]; 2
    // (both slots): K tiles read; 1: the others
    constexpr int N4 = 6, N2 = N4 + KS, NB = N2 + 2 + 2 + 4 + 3 + 3 * KS + 1;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bP = bars, *const bL = bars + 4, *const eK = bars + N4, *const bQ = bars + N2, *const bS = bQ + 2,
                    *const bF = bS + 2, *const bE = bF + 4, *const bK = bE + 3, *const bV = bK + KS, *const eV = bV + KS,
                    *const bT = eV + KS;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;
    __shared__ float2 s_ml[2 * kLpRows];   // (split) a row's reference and sum
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < NB) {
        mbar_init(&bars[tid], tid < N4 ? 4 : tid < N2 ? 2 : 1);
        fence_mbar_init();
    }
    if (tid == 0) s_abort = 0;
    if (warp == 0) tc_alloc(&s_taddr, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    kivi_after_previous();
    const uint32_t taddr = s_taddr;
    const volatile int *abort = &s_abort;
    bool ok = true;
    // the tiles that each slot sees (none: a slot without rows), of this CTA's: x0 on
    const int last1 = min(row0 + 2 * kLpRows, n) - 1, last0 = min(row0 + kLpRows, n) - 1;
    const int all0 = (T + last0) / kLpKeys + 1, all1 = n > row0 + kLpRows ? (T + last1) / kLpKeys + 1 : 0;
    const int share = (max(all0, all1) + a.split - 1) / a.split, x0 = rank * share;
    const int nx0 = max(min(all0 - x0, share), 0), nx1 = max(min(all1 - x0, share), 0), nx = max(nx0, nx1);

    if (warp == 8 || warp == 9) {
        // ---- S = Q K^T of slot e ----
        const int e = __shfl_sync(kFull, warp - 8, 0), mine = e ? nx1 : nx0;
        constexpr uint32_t ID = tc_idesc_f16(kLpRows, kLpKeys, 0);
        CkRing t;
        const uint64_t dq = tc_desc_sw(sQ + e * kLpQ, 16, 1024), dk = tc_desc_sw(sK, 16, 1024);
        for (int x = 0; x < nx && ok; ++x, t.next(KS)) {
            ok = __all_sync(kFull, mbar_wait_ab(&bK[t.s], t.p, abort));
            if (!ok) break;
            if (x >= mine) {   // this slot sees none of the tile: it releases it, once it is in (a phase an arrival)
                if (lane == 0) mbar_arrive(&eK[t.s]);
                continue;
            }
            ok = (x > 0 || mbar_wait_ab(&bQ[e], 0u, abort)) && (x == 0 || mbar_wait_ab(&bL[e], (unsigned)(x - 1) & 1u, abort));
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            tc_fence_after();
            const uint64_t d = dk + (uint32_t)(t.s * (kLpK >> 4));
#pragma unroll
            for (int c = 0; c < kLpQK / 16; ++c)
                tc_mma_f16_w(taddr + 256 * e, dq + (((c >> 2) * kLpQs + (c & 3) * 32) >> 4),
                             d + (((c >> 2) * kLpKs + (c & 3) * 32) >> 4), ID, c > 0);
            tc_commit_w(&bS[e]);
            tc_commit_w(&eK[t.s]);
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(a.status, KIVI_FLAG_WAIT);
        }
        // every MMA and commit has landed before shared memory is given up (bounded)
        tc_commit_w(&bE[e]);
        mbar_wait(&bE[e], 0u);
        __syncwarp();
    } else if (warp == 10) {
        // ---- O += P V ----
        constexpr uint32_t ID = tc_idesc_f16(kLpRows, kLatHead, 1);
        CkRing t;
        const uint64_t dv = tc_desc_sw(sV, kLpKs, 1024);
        for (int x = 0; x < nx && ok; ++x, t.next(KS)) {
            const uint64_t d = dv + (uint32_t)(t.s * (kLpV >> 4));
            ok = __all_sync(kFull, mbar_wait_ab(&bV[t.s], t.p, abort));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!ok || x >= (e ? nx1 : nx0)) continue;
                const int b = x & 1;
                ok = __all_sync(kFull, mbar_wait_ab(&bP[2 * e + b], (unsigned)(x >> 1) & 1u, abort));
                if (!ok) continue;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kLpKeys / 16; ++c)
                    tc_mma_f16_ta_w(taddr + 256 * e + 128, taddr + 256 * e + 64 + 32 * b + 8 * c, d + ((2048 * c) >> 4), ID,
                                    x > 0 || c > 0);
                tc_commit_w(&bF[2 * e + b]);
            }
            if (ok) tc_commit_w(&eV[t.s]);
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(a.status, KIVI_FLAG_WAIT);
        }
        tc_commit_w(&bE[2]);
        mbar_wait(&bE[2], 0u);
        __syncwarp();
    } else if (warp == 11) {
        // ---- copies ----
        const int q0 = pair * a.n_stride, k0 = pair * a.s_stride, S = T + n;   // the head's first rows; tokens
        if (lane == 0)
            for (int e = 0; e < 2; ++e) {
                if ((e ? nx1 : nx0) == 0) continue;
                mbar_expect_tx(&bQ[e], kLpQ);
                for (int c = 0; c < 3; ++c)
                    tma_sw(sQ + e * kLpQ + c * kLpQs, c < 2 ? &tmQn : &tmQr, c < 2 ? 64 * c : 0, q0 + row0 + e * kLpRows, &bQ[e]);
            }
        __syncwarp();
        CkRing t;
        int ck = 0, cv = 0;   // tiles asked for
        for (int x = 0; x < nx && ok; ++x, t.next(KS)) {
            const int tb = (x0 + x) * kLpKeys;
            if (lane == 0) {
                ok = x < KS || mbar_wait_ab(&eK[t.s], t.p ^ 1u, abort);
                if (ok) {
                    mbar_expect_tx(&bK[t.s], kLpK);
                    for (int c = 0; c < 2; ++c) tma_sw(sK + t.s * kLpK + c * kLpKs, &tmK, 64 * c, k0 + tb, &bK[t.s]);
                    tma_sw(sK + t.s * kLpK + 2 * kLpKs, &tmKr, 0, i * a.s_stride + tb, &bK[t.s]);
                    ++ck;
                    ok = x < KS || mbar_wait_ab(&eV[t.s], t.p ^ 1u, abort);
                }
                if (ok) {
                    // (the last tile's rows behind the sequence are zeroed first)
                    uint64_t *const bar = tb + kLpKeys > S ? bT : &bV[t.s];
                    mbar_expect_tx(bar, kLpV);
                    for (int c = 0; c < 2; ++c) tma_sw(sV + t.s * kLpV + c * kLpKs, &tmV, 64 * c, k0 + tb, bar);
                    ++cv;
                }
            }
            ok = __all_sync(kFull, ok);
            if (ok && tb + kLpKeys > S) {
                ok = __all_sync(kFull, mbar_wait_ab(bT, 0u, abort));
                if (ok) {
                    const int c16 = (tb + kLpKeys - S) * 8;   // 16-byte chunks of 64 channels
                    for (int y = lane; y < 2 * c16; y += 32)
                        *reinterpret_cast<uint4 *>(sV + t.s * kLpV + (y / c16) * kLpKs + (S - tb) * 128 + y % c16 * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bV[t.s]);
                }
            }
        }
        if (lane == 0) {
            if (!ok) {
                s_abort = 1;
                atomicOr(a.status, KIVI_FLAG_WAIT);
            }
            // every copy has landed before shared memory is given up (bounded)
            if (nx0) mbar_wait(&bQ[0], 0u);
            if (nx1) mbar_wait(&bQ[1], 0u);
            for (int y = max(0, ck - KS); y < ck; ++y) mbar_wait(&bK[y % KS], (unsigned)(y / KS) & 1u);
            for (int y = max(0, cv - KS); y < cv; ++y) {
                const bool tail = (x0 + y + 1) * kLpKeys > S;
                mbar_wait(tail ? bT : &bV[y % KS], tail ? 0u : (unsigned)(y / KS) & 1u);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax ----
        const int slot = tid / kLpRows, srow = row0 + slot * kLpRows, pos = T + srow + tid % kLpRows;
        const int mine = slot ? nx1 : nx0;
        const uint32_t tS = taddr + 256 * slot + ((uint32_t)(32 * (warp & 3)) << 16), tO = tS + 128;
        float ref = -INFINITY, lsum = 0.f;   // the row's reference less the lift (log2; -inf: nothing yet), the weights' sum
        for (int x = 0; x < mine; ++x) {
            const int b = x & 1, key0 = (x0 + x) * kLpKeys;
            ok = __all_sync(kFull, mbar_wait_ab(&bS[slot], (unsigned)x & 1u, abort));
            if (!ok) break;
            tc_fence_after();
            uint32_t r[2][32];
            tc_ld32(tS, r[0]);
            tc_ld32(tS + 32, r[1]);
            tc_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bL[slot]);
            const bool pf = x < 2 || mbar_test(&bF[2 * slot + b], (unsigned)((x >> 1) + 1) & 1u);
            if (key0 + kLpKeys - 1 > T + srow) {   // some row of the slot does not see the whole tile
                const uint32_t h0 = ck_above(pos - key0), h1 = ck_above(pos - key0 - 32);
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
            const bool grow = mx != -INFINITY && (ref == -INFINITY || fmaf(mx, a.sl2, -ref) > kCkLift + kCkLag);
            const float up = fmaf(mx, a.sl2, -kCkLift);
            const float alpha = grow && ref != -INFINITY ? ex2(ref - up) : 1.f;
            if (grow) ref = up;
            const float ms = ref == -INFINITY ? 0.f : ref;
            const unsigned long long sc2 = lp_f2(a.sl2, a.sl2), ms2 = lp_f2(-ms, -ms);
            unsigned long long l2[4] = {0ull, 0ull, 0ull, 0ull};
            uint32_t pw[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                float y0, y1;
                lp_f2(lp_fma2(lp_f2(__uint_as_float(r[c >> 4][2 * c & 31]), __uint_as_float(r[c >> 4][(2 * c & 31) + 1])), sc2,
                              ms2), y0, y1);
                y0 = ex2(y0);
                y1 = ex2(y1);
                l2[c & 3] = lp_add2(l2[c & 3], lp_f2(y0, y1));
                pw[c] = ck_pack(y0, y1);
            }
            float l0, l1;
            lp_f2(lp_add2(lp_add2(l2[0], l2[1]), lp_add2(l2[2], l2[3])), l0, l1);
            lsum = lsum * alpha + (l0 + l1);
            if (x > 0 && __any_sync(kFull, alpha != 1.f)) {   // rescale O, once P V of tile x - 1 is in
                ok = __all_sync(kFull, mbar_wait_ab(&bF[2 * slot + (b ^ 1)], (unsigned)((x - 1) >> 1) & 1u, abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < kLatHead; c0 += 32) {
                    uint32_t o[32];
                    tc_ld32(tO + c0, o);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                    tc_st32(tO + c0, o);
                }
            }
            ok = __all_sync(kFull, pf || mbar_wait_ab(&bF[2 * slot + b], (unsigned)((x >> 1) + 1) & 1u, abort));
            if (!ok) break;
            tc_fence_after();
            tc_st32(tS + 64 + 32 * b, pw);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bP[2 * slot + b]);
        }
        for (int y = max(mine - 2, 0); y < mine && ok; ++y)
            ok = __all_sync(kFull, mbar_wait_ab(&bF[2 * slot + (y & 1)], (unsigned)(y >> 1) & 1u, abort));
        if (a.split > 1) {
            s_ml[tid] = make_float2(ref, lsum);
        } else if (ok && mine > 0) {
            tc_fence_after();
            // 32 columns at a time through shared memory (Q's, which the slot's
            // products have read; 16-byte chunk c of row r at chunk c ^ (r / 2
            // mod 4) of it: no bank conflicts): a store covers 64 consecutive
            // bytes of 8 rows
            const float inv = 1.f / lsum;
            unsigned char *st = sQ + slot * kLpQ + (warp & 3) * (32 * 64);
            const int q8 = lane >> 2, c4 = lane & 3, row32 = srow + 32 * (warp & 3);
            __half *dst = a.out + ((size_t)pair * a.n_stride + row32) * kLatHead + 8 * c4;
#pragma unroll 1
            for (int c0 = 0; c0 < kLatHead; c0 += 32) {
                uint32_t o[32];
                tc_ld32(tO + c0, o);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4 *>(st + lane * 64 + ((c ^ (lane >> 1)) & 3) * 16) =
                        make_uint4(ck_pack(__uint_as_float(o[8 * c]) * inv, __uint_as_float(o[8 * c + 1]) * inv),
                                   ck_pack(__uint_as_float(o[8 * c + 2]) * inv, __uint_as_float(o[8 * c + 3]) * inv),
                                   ck_pack(__uint_as_float(o[8 * c + 4]) * inv, __uint_as_float(o[8 * c + 5]) * inv),
                                   ck_pack(__uint_as_float(o[8 * c + 6]) * inv, __uint_as_float(o[8 * c + 7]) * inv));
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int q = 8 * k + q8;
                    const uint4 v = *reinterpret_cast<const uint4 *>(st + q * 64 + ((c4 ^ (q >> 1)) & 3) * 16);
                    if (row32 + q < n) *reinterpret_cast<uint4 *>(dst + (size_t)q * kLatHead + c0) = v;
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(a.status, KIVI_FLAG_WAIT);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (a.split > 1) {   // (every product has ended and every copy landed: shared memory is free)
        cg::cluster_group cl = cg::this_cluster();
        float4 *const part = reinterpret_cast<float4 *>(smem);   // [row][32 chunks, chunk c at c ^ (row mod 8): no bank conflicts]
        if (warp < 8 && (warp < 4 ? nx0 : nx1) > 0) {
            tc_fence_after();
            const uint32_t tO = taddr + 256 * (warp >> 2) + ((uint32_t)(32 * (warp & 3)) << 16) + 128;
#pragma unroll 1
            for (int c0 = 0; c0 < kLatHead; c0 += 32) {
                uint32_t o[32];
                tc_ld32(tO + c0, o);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    part[tid * 32 + ((c0 / 4 + c) ^ (tid & 7))] =
                        make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]), __uint_as_float(o[4 * c + 2]),
                                    __uint_as_float(o[4 * c + 3]));
            }
            tc_fence_before();
        }
        cl.sync();
        // a warp joins a row: weights 2^(ref_k - M), M the largest reference
        const int rows = (2 * kLpRows + a.split - 1) / a.split, end = min(min((rank + 1) * rows, 2 * kLpRows), n - row0);
        for (int q = rank * rows + warp; q < end; q += kLpThreads / 32) {
            const float2 ml = lane < a.split ? *cl.map_shared_rank(&s_ml[q], lane) : make_float2(-INFINITY, 0.f);
            float M = ml.x;
#pragma unroll
            for (int o = kLpMaxSplit / 2; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
            const float mine = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);   // (0: the share holds nothing that the row sees)
            float L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int k = 0; k < a.split; ++k) {
                const float w = __shfl_sync(kFull, mine, k);
                L = fmaf(w, __shfl_sync(kFull, ml.y, k), L);
                if (w == 0.f) continue;
                const float4 y = cl.map_shared_rank(part, k)[q * 32 + (lane ^ (q & 7))];
                acc.x = fmaf(w, y.x, acc.x);
                acc.y = fmaf(w, y.y, acc.y);
                acc.z = fmaf(w, y.z, acc.z);
                acc.w = fmaf(w, y.w, acc.w);
            }
            const float inv = 1.f / L;
            *reinterpret_cast<uint2 *>(a.out + ((size_t)pair * a.n_stride + row0 + q) * kLatHead + 4 * lane) =
                make_uint2(ck_pack(acc.x * inv, acc.y * inv), ck_pack(acc.z * inv, acc.w * inv));
        }
        cl.sync();   // the others have read this CTA's sums
    }
    if (warp == 0) tc_dealloc(taddr, 512);
}

// Clusters of c CTAs that the device holds at once (0: none).
int clusters(int c, int device) {
    static std::atomic<int> known[64][kLpMaxSplit + 1];   // one more than they are
    std::atomic<int> *const slot = device < 64 ? &known[device][c] : nullptr;
    int v = slot ? slot->load(std::memory_order_relaxed) : 0;
    if (v > 0) return v - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = kLpSmem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)c;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&v, latent_prompt_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        v = 0;
    }
    if (slot) slot->store(v + 1, std::memory_order_relaxed);
    return v;
}
// CTAs a row tile (of `tiles`, up to nx key tiles each): what ends first, where a
// device full of clusters follows another.
int shares(long long tiles, int nx, int device, int sms) {
    int best = 1;
    long long least = (tiles + sms - 1) / sms * nx;
    for (int c = 2; c <= kLpMaxSplit && tiles * c <= sms; ++c) {
        const int at_once = clusters(c, device);
        if (at_once < 1) continue;
        const long long t = (tiles + at_once - 1) / at_once * ((nx + c - 1) / c + kLpJoin);
        if (t < least) {
            least = t;
            best = c;
        }
    }
    return best;
}

kivi_status fail(kivi_status s, const char *msg) {
    kivi_set_last_error(msg);
    return s;
}

}  // namespace

// n[i] queries behind T[i] tokens (T null: none)
kivi_status kivi_latent_expanded_to(unsigned *status, const void *q, const void *q_rope, const void *K, const void *Kr,
                                    const void *V, int b, int h, const int32_t *T, const int32_t *n, int n_stride,
                                    int s_stride, float scale, void *out, kivi_stream_t stream) {
    if (b < 1 || h < 1 || n_stride < 0 || s_stride < 0) return fail(KIVI_ERR_INVALID_ARG, "sizes must be positive");
    if (b > KIVI_MAX_BATCH) return fail(KIVI_ERR_UNSUPPORTED, "b above 1024");
    if (h > 1024) return fail(KIVI_ERR_UNSUPPORTED, "more than 1024 heads");
    if (n_stride > (1 << 26) || s_stride > (1 << 26) || (long long)b * h * n_stride >= (1LL << 31) ||
        (long long)b * h * s_stride >= (1LL << 31))
        return fail(KIVI_ERR_UNSUPPORTED, "a stride above 2^26, or b h times it not below 2^31");
    if (!(scale > 0.f && scale - scale == 0.f)) return fail(KIVI_ERR_INVALID_ARG, "scale must be positive and finite");
    if (!n) return fail(KIVI_ERR_INVALID_ARG, "the counts are null");
    PromptArgs a;
    int maxn = 0;
    for (int i = 0; i < b; ++i) {
        a.n[i] = n[i];
        a.T[i] = T ? T[i] : 0;
        if (n[i] < 0 || n[i] > n_stride) return fail(KIVI_ERR_INVALID_ARG, "a count outside its stride");
        if (n[i] > 0 && (a.T[i] < 0 || a.T[i] > s_stride - n[i]))
            return fail(KIVI_ERR_INVALID_ARG, "tokens before the queries negative, or past the keys' stride");
        maxn = n[i] > maxn ? n[i] : maxn;
    }
    if (maxn == 0) return KIVI_OK;
    if (!q || !q_rope || !K || !Kr || !V || !out) return fail(KIVI_ERR_INVALID_ARG, "a tensor pointer is null");
    if (((uintptr_t)q | (uintptr_t)q_rope | (uintptr_t)K | (uintptr_t)Kr | (uintptr_t)V | (uintptr_t)out) & 15u)
        return fail(KIVI_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    a.out = (__half *)out;
    a.b = b;
    a.h = h;
    a.n_stride = n_stride;
    a.s_stride = s_stride;
    a.mt = (maxn + 2 * kLpRows - 1) / (2 * kLpRows);
    a.sl2 = scale * 1.4426950408889634f;
    long long tiles = 0;
    int longest = 0;   // row tiles; tokens
    for (int i = 0; i < b; ++i)
        if (n[i] > 0) {
            tiles += (long long)(n[i] + 2 * kLpRows - 1) / (2 * kLpRows) * h;
            longest = a.T[i] + n[i] > longest ? a.T[i] + n[i] : longest;
        }
    if ((long long)a.mt * b * h > INT_MAX / kLpMaxSplit) return fail(KIVI_ERR_UNSUPPORTED, "more than 2^28 row tiles");
    KiviDeviceInfo info;
    if (!kivi_device_info(&info)) return fail(KIVI_ERR_CUDA, "no status word on the current device");
    a.status = status ? status : info.status;
    const long long rows = (long long)b * h * n_stride, keys = (long long)b * h * s_stride;
    CUtensorMap tq, tqr, tk, tkr, tv;
    cudaError_t e = make_sw_map(&tq, (const __half *)q, rows, kLatHead, kLpRows);
    if (e == cudaSuccess) e = make_sw_map(&tqr, (const __half *)q_rope, rows, kLatRope, kLpRows);
    if (e == cudaSuccess) e = make_sw_map(&tk, (const __half *)K, keys, kLatHead, kLpKeys);
    if (e == cudaSuccess) e = make_sw_map(&tkr, (const __half *)Kr, (long long)b * s_stride, kLatRope, kLpKeys);
    if (e == cudaSuccess) e = make_sw_map(&tv, (const __half *)V, keys, kLatHead, kLpKeys);
    static std::atomic<uint64_t> done;
    if (e == cudaSuccess) e = kivi_allow_smem(latent_prompt_kernel, kLpSmem, info.device, done);
    if (e == cudaSuccess) a.split = shares(tiles, (longest + kLpKeys - 1) / kLpKeys, info.device, info.sms);
    if (e != cudaSuccess) return fail(KIVI_ERR_CUDA, cudaGetErrorString(e));
    e = kivi_launch_after(latent_prompt_kernel, dim3((unsigned)(a.mt * b * h * a.split)), kLpThreads, kLpSmem,
                          (cudaStream_t)stream, a.split, tq, tqr, tk, tkr, tv, a);
    return e == cudaSuccess ? KIVI_OK : fail(KIVI_ERR_CUDA, cudaGetErrorString(e));
}

extern "C" kivi_status kivi_latent_prompt_attn(const void *q, const void *q_rope, const void *K, const void *Kr,
                                               const void *V, int b, int h, const int32_t *t, int t_stride, float scale,
                                               void *out, kivi_stream_t stream) {
    kivi_set_last_error("");
    return kivi_latent_expanded_to(nullptr, q, q_rope, K, Kr, V, b, h, nullptr, t, t_stride, t_stride, scale, out, stream);
}

extern "C" kivi_status kivi_latent_expanded_attn(const void *q, const void *q_rope, const void *K, const void *Kr,
                                                 const void *V, int b, int h, const int32_t *T, const int32_t *n,
                                                 int n_stride, int s_stride, float scale, void *out,
                                                 kivi_stream_t stream) {
    kivi_set_last_error("");
    if (!T) return fail(KIVI_ERR_INVALID_ARG, "T is null");
    return kivi_latent_expanded_to(nullptr, q, q_rope, K, Kr, V, b, h, T, n, n_stride, s_stride, scale, out, stream);
}
