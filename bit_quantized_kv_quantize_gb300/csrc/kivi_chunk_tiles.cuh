// kivi_chunk_tiles.cuh -- what the chunk attention's kernels share: packed
// records to fp16 tiles, the walk over a CTA's share of the work, and the
// join of partial results.
#pragma once
#include <cuda_fp16.h>

#include "kivi_async.cuh"
#include "kivi_chunk.cuh"
#include "kivi_internal.cuh"
#include "kivi_mma.cuh"
#include "kivi_unpack.cuh"

namespace {

constexpr int kCkDqGroup = 4;    // warps that restore a record together
constexpr unsigned kFull = 0xffffffffu;
constexpr int kJoinRows = 16;    // rows of a row tile that a block joins
// Weights are taken 2^7 above their row's reference.  In fp16 a weight loses
// all below 2^-25; lifted, that is 2^-32 of the reference's own weight, and a
// score 2^8 above the reference (kCkLag: from there on it is raised) still is
// a finite 2^15.  Many tokens far below one sink then keep their share: 32k of
// them 17.5 below it came out 8e-4 too small without the lift.
constexpr float kCkLift = 7.f, kCkLag = 8.f;   // log2

__device__ __forceinline__ uint32_t ck_pack(float lo, float hi) {
    return h2u(__floats2half2_rn(lo, hi));
}
// s code + z of two values, the code from off + code (exact)
__device__ __forceinline__ uint32_t ck_affine(uint32_t x, float off, uint32_t s, uint32_t z) {
    return h2u(__hfma2(__hsub2(u2h(x), __float2half2_rn(off)), u2h(s), u2h(z)));
}


// K^ of a record's 64 tokens: into 64 rows of a chunk-major tile
// [TK tokens][D] (tile: the first of them): 16-byte chunk c of row r at byte
// c TK 16 + r 16.  Warp w of the kCkDqGroup takes the
// 16-channel steps w, w + kCkDqGroup, ...; a lane's half2 (two channels of one token) are
// the lanes t = 0..3 of one 16-byte chunk: 128 consecutive bytes a store.
template <int D, int KB, int TK>
__device__ __forceinline__ void dequant_keys(unsigned char *tile, const unsigned char *rec, int off_ksz, int lgG,
                                             int w) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const __half *ksz = reinterpret_cast<const __half *>(rec + off_ksz) + tq * (D / 4);
    unsigned char *dst = tile + gq * 16 + tq * 4;
    constexpr int NW = KB / 2;   // words of a channel pair
    // one 16-channel step a turn, not unrolled (see dequant_values)
#pragma unroll 1
    for (int j = w; j < D / 16; j += kCkDqGroup) {
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
        unsigned char *p = dst + (size_t)(2 * j) * (TK * 16);
#pragma unroll
        for (int pos = 0; pos < 8; ++pos) {
            const int wi = KB == 2 ? 0 : pos >> 2, r = KB == 2 ? pos : pos & 3;
            const float off = slot_offset<KB, true>(r);
            const uint2 sc = sv[pos >> 1], z = zv[pos >> 1];
            *reinterpret_cast<uint32_t *>(p + pos * 128) = ck_affine(unpack<KB, true>(W[wi], r), off, sc.x, z.x);
            *reinterpret_cast<uint32_t *>(p + TK * 16 + pos * 128) =
                ck_affine(unpack<KB, true>(W[NW + wi], r), off, sc.y, z.y);
        }
    }
}

// V^ of a record's 64 tokens, transposed: into 64 tokens of a chunk-major tile
// [D channels][tokens] (tile: the first of them): tokens 8 k .. 8 k + 7 of
// channel c at byte k D 16 + c 16.  Warp w
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

// The same by the cache's bit widths, for tiles that also hold fp16 tokens:
// out of line, as other code that does not run every tile (with a role a
// warp, the loops that do must share the instruction cache).
template <int D, int TK>
__device__ __noinline__ void dequant_keys_cold(unsigned char *tile, const unsigned char *rec, int bits, int off_ksz,
                                               int lgG, int w) {
    if (bits == 2) dequant_keys<D, 2, TK>(tile, rec, off_ksz, lgG, w);
    else dequant_keys<D, 4, TK>(tile, rec, off_ksz, lgG, w);
}
template <int D>
__device__ __noinline__ void dequant_values_cold(unsigned char *tile, const unsigned char *rec, int bits, int off_vc,
                                                 int off_vsz, int lgG, int w) {
    if (bits == 2) dequant_values<D, 2>(tile, rec, off_vc, off_vsz, lgG, w);
    else dequant_values<D, 4>(tile, rec, off_vc, off_vsz, lgG, w);
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
    __device__ __forceinline__ void skip(int k, int n) {
        for (s += k; s >= n; s -= n) p ^= 1u;
    }
};

// A CTA's share of one row tile.
struct CkSeg {
    int i, j, m;     // sequence, kv head, row tile
    int T, n;        // cached tokens, chunk tokens
    int row0, nrows; // first row, rows of (i, j)
    int nb, nt;      // the row tile's blocks and key tiles
    int x0, nx;      // the CTA's key tiles
    BlockList bl;
    // first token of the CTA's tile x (tiles of one block)
    __device__ __forceinline__ int key0(int x) const { return bl.phys(x0 + x) * KIVI_KBLK; }
};

// Walks a CTA's units: every warp runs the same walk.  LEAD: the units of a row
// tile's fixed cost.
template <int LEAD = kCkLead>
struct CkWalk {
    int left;        // units left
    int i, m, j, o;  // where they begin
    __device__ __forceinline__ void start(const ChunkArgs &a, int c) {
        const ChunkPos &p = a.cta[c];
        left = (int)(a.cta[c + 1].u - p.u);
        i = p.i;
        m = p.m;
        j = p.j;
        o = p.o;
    }
    // the next segment with tiles; false at the end
    __device__ __forceinline__ bool next(const KiviGeom &g, const ChunkArgs &a, CkSeg &s) {
        while (left > 0) {
            const int nb = chunk_blocks(a, i, m), nt = a.tile_blocks == 2 ? (nb + 1) >> 1 : nb;
            const int w = LEAD + nt, o1 = min(w, o + left);
            const int x0 = max(o - LEAD, 0), x1 = max(o1 - LEAD, 0);
            s.i = i;
            s.j = j;
            s.m = m;
            s.T = a.T[i];
            s.n = a.n[i];
            s.row0 = m * a.tile_rows;
            s.nrows = s.n * a.hg;
            s.nb = nb;
            s.nt = nt;
            s.x0 = x0;
            s.nx = x1 - x0;
            s.bl = visible_blocks(a.vis, s.T + chunk_div(a, s.row0));
            left -= o1 - o;
            o = 0;
            if (o1 == w && ++j == g.h) {
                j = 0;
                if (++m * a.tile_rows >= s.nrows) {
                    m = 0;
                    do ++i; while (i < g.b && a.n[i] == 0);
                }
            }
            if (x1 > x0) return true;
        }
        return false;
    }
};

// Which of 16 rows (r, e), the first of them head e0 of hg at position p0, do
// not see token `key`: bit c for row c.
__device__ __noinline__ uint32_t ck_hidden16(int key, int p0, int e0, int hg, int window, int sinks) {
    uint32_t m = 0;
    int p = p0, e = e0;
    for (int c = 0; c < 16; ++c) {
        if (key > p || (window > 0 && key <= p - window && key >= sinks)) m |= 1u << c;
        if (++e == hg) {
            e = 0;
            ++p;
        }
    }
    return m;
}
// bit c for c > x
__device__ __forceinline__ uint32_t ck_above(int x) { return x < 0 ? 0xffffffffu : x >= 31 ? 0u : 0xfffffffeu << x; }
// Which of the 32 tokens key0, key0 + 1, ... the row at position p does not
// see: bit c for token key0 + c.
__device__ __forceinline__ uint32_t ck_hidden32(int key0, int p, int window, int sinks) {
    const uint32_t future = ck_above(p - key0);
    return window > 0 ? future | (~ck_above(p - window - key0) & ck_above(sinks - 1 - key0)) : future;
}

// Joins the partials of the row tiles that CTA boundaries cut, a block per
// cut row tile and kJoinRows of its rows (a warp takes rows w, w + 8):
// weights 2^(m_k - M), M the largest m.  A block finds its row tile from a CTA
// boundary; the first boundary behind the row tile's first key tile owns it.
template <int D>
__global__ void __launch_bounds__(256)
    chunk_join_kernel(__half *__restrict__ O, const __grid_constant__ ChunkArgs a) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nq = a.tile_rows / kJoinRows, c = blockIdx.x / nq + 1, r0 = blockIdx.x % nq * kJoinRows;
    const ChunkPos &p = a.cta[c];
    if (p.o <= kCkLead) return;   // CTA c starts with a row tile of its own
    const int i = p.i, m = p.m, hg = a.hg;
    const long long first = p.u - p.o + kCkLead;                         // the unit of its first key tile
    if (a.cta[c - 1].u > first) return;                                  // an earlier boundary owns it
    const long long end = first + chunk_tiles(a, i, m);
    int c1 = c;                                                          // the last CTA with its tiles
    while (a.cta[c1 + 1].u < end) ++c1;
    // CTA c - 1 holds the first key tile and runs into it (slot 2 c + 1), the
    // others start in it (slot 2 c)
    const int c0 = c - 1;
    const float2 *ml = reinterpret_cast<const float2 *>(a.ml);
    const int nrows = min(a.n[i] * hg - m * a.tile_rows, a.tile_rows);
    for (int r = r0 + warp; r < min(nrows, r0 + kJoinRows); r += 8) {
        auto part = [&](int k) { return (size_t)(2 * k + (k == c0 ? 1 : 0)) * a.tile_rows + r; };
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
        const int row = m * a.tile_rows + r, tok = chunk_div(a, row);
        __half *dst = O + (((size_t)i * a.hq + p.j * hg + row - tok * hg) * a.n_stride + tok) * D + lane * V;
#pragma unroll
        for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t *>(dst + v) = ck_pack(acc[v] * inv, acc[v + 1] * inv);
    }
}

}  // namespace
