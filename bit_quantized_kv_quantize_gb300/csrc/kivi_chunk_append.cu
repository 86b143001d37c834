// kivi_chunk_append.cu -- append a chunk of new tokens to every sequence.
//
// Method: n one-token appends ("Literature audit -- Group 2", section 1
// KIVI, core algorithm items 1-4) leave the keys [Tqk, Tqk') and values
// [Tqv, Tqv') newly quantized, with Tqk' = R floor((T + n - 1) / R) and
// Tqv' = T + n - R - 1 (if larger), and the last R (R + 1) tokens in the
// windows' slots.  That depends on the end only, so the chunk is packed in
// one pass, from the window rows (tokens below T) and the chunk's, bitwise
// as the one-token appends would.
//
// Two launches: the windows' old rows are still read by the first (one CTA the
// keys, and one the values, of a block of max(64, G) tokens: whole key groups
// and whole 64-token records, so no word has two writers), the second
// overwrites them and writes the counters.  Bound: the quantizer's instructions
// in a CTA's few passes (bytes: a chunk token of a kv head reads 4 d and writes
// its packed 0.5-1.3 d).  2048 tokens of 8 heads 23 us, 512 tokens of 8
// sequences 32 us (a CTA for both: 33 and 51 us).
#include "kivi_append_impl.cuh"
#include "kivi_chunk.cuh"

namespace {

constexpr int kApThreads = 256;

__host__ __device__ __forceinline__ int span_of(const KiviGeom &g) { return g.G > KIVI_KBLK ? g.G : KIVI_KBLK; }

__global__ void __launch_bounds__(kApThreads)
    chunk_pack_kernel(KiviGeom g, KiviDev dv, const __half *__restrict__ Kn, const __half *__restrict__ Vn,
                      const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int i = blockIdx.z, j = blockIdx.y, d = g.d, R = g.R, CA = span_of(g);
    const int T = a.T[i], Tqk = a.Tqk[i], Tqv = a.Tqv[i], n = a.n[i];
    const int Tqk1 = chunk_tqk(T, Tqk, n, R), Tqv1 = chunk_tqv(T, Tqv, n, R);
    // the CTA's tokens [cs, cs + CA), their keys or values
    const int cs = (min(Tqk, Tqv) / CA + (blockIdx.x >> 1)) * CA;
    const bool keys = !(blockIdx.x & 1);
    const int ka = max(cs, Tqk), kz = min(cs + CA, Tqk1), va = max(cs, Tqv), vz = min(cs + CA, Tqv1);
    __half *xs = reinterpret_cast<__half *>(smem);   // [CA][d]
    float *s_f = reinterpret_cast<float *>(smem + (size_t)CA * d * 2);
    const int nv = d / 8, lgv = __ffs(nv) - 1, lgG = __ffs(g.G) - 1;
    // rows of tokens [x, y): below T from the window, the others from the chunk
    auto stage = [&](const __half *win, int ring, const __half *chk, int x, int y) {
        chk += ((size_t)i * g.h + j) * a.n_stride * d;
        for (int e = threadIdx.x; e < (y - x) * nv; e += kApThreads) {
            const int tau = x + (e >> lgv), c8 = e & (nv - 1);
            const __half *src = tau < T ? win + (size_t)(tau % ring) * d : chk + (size_t)(tau - T) * d;
            reinterpret_cast<uint4 *>(xs + (size_t)(tau - cs) * d)[c8] = reinterpret_cast<const uint4 *>(src)[c8];
        }
        __syncthreads();
    };
    if (keys && ka < kz) {
        stage(dv.Kf + kf_slice(g, i, j), R, Kn, ka, kz);
        pack_key_round(g, dv, i, j, xs, s_f, cs, CA, ka, kz, Tqk);
    }
    if (!keys && va < vz) {
        stage(dv.Vf + vf_slice(g, i, j), R + 1, Vn, va, vz);
        const int ngi = d >> lgG, lgn = __ffs(ngi) - 1;
        float *s_s = s_f, *s_z = s_s + CA * ngi, *s_r = s_z + CA * ngi;   // [token][group]
        // value blocks opened here: cleared, so untouched fields read zero
        for (int vb = (va + KIVI_VBLK - 1) / KIVI_VBLK; vb * KIVI_VBLK < vz; ++vb) {
            uint32_t *vc = vc_words(g, dv.blk, i, j, vb);
            __half *vsz = vsz_halves(g, dv.blk, i, j, vb);
            for (int e = threadIdx.x; e < g.vc_blk; e += kApThreads) vc[e] = 0u;
            for (int e = threadIdx.x; e < g.vsz_blk; e += kApThreads) vsz[e] = __float2half_rn(0.f);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < (vz - va) << lgn; e += kApThreads) {
            const int tau = va + (e >> lgn), gi = e & (ngi - 1), nc = g.G / 8;
            const uint4 *x = reinterpret_cast<const uint4 *>(xs + (size_t)(tau - cs) * d + gi * g.G);
            float mn = INFINITY, mx = -INFINITY;
            for (int k = 0; k < nc; ++k) {   // 8 channels, from another one each thread (bank conflicts)
                const uint4 v = x[(k + 2 * tau + (gi >> 1)) & (nc - 1)];
                const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[m]));
                    mn = fminf(mn, fminf(y.x, y.y));
                    mx = fmaxf(mx, fmaxf(y.x, y.y));
                }
            }
            const QParams p = qparams(mn, mx, g.vbits);
            __half *vsz = vsz_halves(g, dv.blk, i, j, tau / KIVI_VBLK);
            vsz[vsz_in_block(g, tau, gi, 0)] = p.s16;
            vsz[vsz_in_block(g, tau, gi, 1)] = p.z16;
            const int q = ((tau - cs) << lgn) + gi;
            s_s[q] = p.sf;
            s_z[q] = p.zf;
            s_r[q] = p.sf == 0.0f ? 0.0f : __frcp_rn(p.sf);
        }
        __syncthreads();
        // a token's 16-bit halves: lane class gg (8) x channel words w (d vbits / 128)
        const int nwv = d * g.vbits / 128, lgw = __ffs(nwv) - 1, cph = 16 / g.vbits, vcs = v_cs(g), lgc = __ffs(vcs) - 1;
        for (int e = threadIdx.x; e < (vz - va) << (3 + lgw); e += kApThreads) {
            const int tau = va + (e >> (3 + lgw)), gg = e & 7, w = (e >> 3) & (nwv - 1), tt = tau % KIVI_VBLK;
            const __half *x = xs + (size_t)(tau - cs) * d;
            uint32_t bits = 0;
            for (int r = 0; r < cph; ++r) {
                const int c = 8 * (w * cph + r) + gg, gi = ((tau - cs) << lgn) + (c >> lgG);
                bits |= qcode_rcp(__half2float(x[c]), s_s[gi], s_z[gi], s_r[gi], g.vbits) << (r * g.vbits);
            }
            const int L = 4 * gg + ((tt & 7) >> 1), u = (tt >> 3) * nwv + w;
            uint32_t *vc = vc_words(g, dv.blk, i, j, tau / KIVI_VBLK);
            reinterpret_cast<uint16_t *>(vc + (size_t)(u >> lgc) * 32 * vcs + (size_t)L * vcs + (u & (vcs - 1)))[tt & 1] =
                (uint16_t)bits;
        }
    }
}

// The last R keys and R + 1 values of the chunk to their window slots, and
// the counters after it.
__global__ void __launch_bounds__(kApThreads)
    chunk_window_kernel(KiviGeom g, KiviDev dv, const __half *__restrict__ Kn, const __half *__restrict__ Vn,
                        const __grid_constant__ ChunkArgs a, int *nxt) {
    const int i = blockIdx.z, j = blockIdx.y, R = g.R, nv = g.d / 8;
    const int T = a.T[i], n = a.n[i];
    const size_t base = ((size_t)i * g.h + j) * a.n_stride * nv;
    uint4 *kw = reinterpret_cast<uint4 *>(dv.Kf + kf_slice(g, i, j));
    uint4 *vw = reinterpret_cast<uint4 *>(dv.Vf + vf_slice(g, i, j));
    const int keep = min(n, R + 1), r0 = n - keep;
    for (int e = blockIdx.x * kApThreads + threadIdx.x; e < keep * nv; e += gridDim.x * kApThreads) {
        const int r = r0 + e / nv, c = e % nv, tau = T + r;
        if (r >= n - R)
            kw[(size_t)(tau % R) * nv + c] = reinterpret_cast<const uint4 *>(Kn)[base + (size_t)r * nv + c];
        vw[(size_t)(tau % (R + 1)) * nv + c] = reinterpret_cast<const uint4 *>(Vn)[base + (size_t)r * nv + c];
    }
    if (j == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        nxt[i] = T + n;
        nxt[g.b + i] = chunk_tqk(T, a.Tqk[i], n, R);
        nxt[2 * g.b + i] = chunk_tqv(T, a.Tqv[i], n, R);
    }
}

}  // namespace

cudaError_t kivi_launch_append_chunk(const KiviGeom &g, const KiviDev &dv, const __half *K, const __half *V,
                                     const ChunkArgs &a, int *nxt, cudaStream_t st) {
    const int CA = span_of(g);
    int blocks = 0, maxn = 0;
    for (int i = 0; i < g.b; ++i) {
        const int k1 = chunk_tqk(a.T[i], a.Tqk[i], a.n[i], g.R), v1 = chunk_tqv(a.T[i], a.Tqv[i], a.n[i], g.R);
        const int lo = a.Tqk[i] < a.Tqv[i] ? a.Tqk[i] : a.Tqv[i], hi = k1 > v1 ? k1 : v1;
        if (k1 > a.Tqk[i] || v1 > a.Tqv[i]) {
            const int c = (hi + CA - 1) / CA - lo / CA;
            blocks = c > blocks ? c : blocks;
        }
        maxn = a.n[i] > maxn ? a.n[i] : maxn;
    }
    const size_t par = 3 * (size_t)(CA / g.G) * g.d, val = 3 * (size_t)CA * (g.d / g.G);   // key, value parameters
    const size_t smem = (size_t)CA * g.d * 2 + (par > val ? par : val) * 4;
    if (blocks > 0) {
        cudaError_t e = cudaFuncSetAttribute(chunk_pack_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        chunk_pack_kernel<<<dim3(2 * blocks, g.h, g.b), kApThreads, smem, st>>>(g, dv, K, V, a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const int keep = maxn < g.R + 1 ? maxn : g.R + 1;
    int gx = (keep * (g.d / 8) + 4 * kApThreads - 1) / (4 * kApThreads);
    if (gx < 1) gx = 1;
    chunk_window_kernel<<<dim3(gx, g.h, g.b), kApThreads, 0, st>>>(g, dv, K, V, a, nxt);
    return cudaGetLastError();
}
