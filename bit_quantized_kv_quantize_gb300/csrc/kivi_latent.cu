// kivi_latent.cu -- the latent cache: its handle, the kernels that fill and
// read it, and the C entry points of latent attention.
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <set>
#include <vector>

#include "../../include/kivi.h"
#include "kivi_latent.cuh"

namespace {

__device__ unsigned g_status;   // of the calls without a handle

// ---------------------------------------------------------------------------
// Append.  Warp x takes new token tau = T + x: to codes where R newer ones follow,
// else into the ring as it is.  The cached tokens that leave the window, [Tq, Tq1)
// below T, are quantized from the ring, each by one warp: that of the new token which
// takes its place, before that is overwritten, or one that has no part in the place
// otherwise.  Where a block is begun, its places behind the last token are set to zero
// (kivi_latent_places.h).
//
// Bound: of single tokens the latency of one round trip, of long fills instructions
// (quantizing r values a token: issue 76 %, HBM 27 %; 2 r + 128 bytes are read a token,
// its codes or 16-bit rows written).  r = 512, 4 bits, R = 128, in a captured graph: a
// token of 64 sequences 3.1 us (3.9 where every one begins a block), 1024 tokens 3.5, a
// fill of 4096 5.1, of 8 x 32767 180 (2.3 TB/s).
// ---------------------------------------------------------------------------
constexpr int kApWarps = 4;

// a token's channels [CH l, CH (l + 1)) as fp16 pairs; CH 8 or 16
template <int CH>
struct LatRow {
    uint4 v[CH / 8];
    // from a row of memory
    __device__ __forceinline__ void load(const __half *row, int lane) {
#pragma unroll
        for (int k = 0; k < CH / 8; ++k) v[k] = *reinterpret_cast<const uint4 *>(row + CH * lane + 8 * k);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < CH / 8; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
    }
    // from, or to, token t of a block of the ring
    __device__ __forceinline__ void load_block(const __half *blk, int t, int lane) {
#pragma unroll
        for (int k = 0; k < CH / 8; ++k)
            v[k] = *reinterpret_cast<const uint4 *>((const char *)blk + lat_at(CH / 8 * lane + k, t, kLatTok));
    }
    __device__ __forceinline__ void store_block(__half *blk, int t, int lane) const {
#pragma unroll
        for (int k = 0; k < CH / 8; ++k)
            *reinterpret_cast<uint4 *>((char *)blk + lat_at(CH / 8 * lane + k, t, kLatTok)) = v[k];
    }
};

// the row as codes, scales and zeros of token t of a record; row: as they restore it
template <int CH, int BITS>
__device__ __forceinline__ void lat_quantize(const LatentGeom &g, unsigned char *rec, int t, LatRow<CH> &row) {
    const int lane = threadIdx.x & 31, gl = g.G / CH;   // lanes a group
    float x[CH];
#pragma unroll
    for (int k = 0; k < CH / 2; ++k) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(row.v)[k];
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
    float mn = x[0], mx = x[0];
#pragma unroll
    for (int k = 1; k < CH; ++k) {
        mn = fminf(mn, x[k]);
        mx = fmaxf(mx, x[k]);
    }
    for (int o = 1; o < gl; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const QParams p = qparams(mn, mx, BITS);
    const float rs = __fdiv_rn(1.f, p.sf);
    if (lane % gl == 0)
        *reinterpret_cast<__half2 *>(rec + g.off_sz + ((lane / gl) * kLatTok + t) * 4) = __halves2half2(p.s16, p.z16);
    constexpr int PW = 32 / BITS, NW = (CH + PW - 1) / PW;   // channels a 32-bit word, words a lane (of 2 bits and 8 channels: half a word)
    uint32_t w[NW];
#pragma unroll
    for (int k = 0; k < NW; ++k) w[k] = 0;
#pragma unroll
    for (int k = 0; k < CH; k += 2) {
        const uint32_t q0 = qcode_rcp(x[k], p.sf, p.zf, rs, BITS), q1 = qcode_rcp(x[k + 1], p.sf, p.zf, rs, BITS);
        w[k / PW] |= (q0 | q1 << 16) << (BITS * ((k % PW) >> 1));
        const __half2 y = __hfma2(__halves2half2(__uint2half_rn(q0), __uint2half_rn(q1)), __half2half2(p.s16), __half2half2(p.z16));
        reinterpret_cast<uint32_t *>(row.v)[k / 2] = *reinterpret_cast<const uint32_t *>(&y);
    }
    if (CH < PW) {   // two lanes share a word
        w[0] <<= BITS * (CH / 2) * (lane & 1);
        w[0] |= __shfl_xor_sync(0xffffffffu, w[0], 1);
        if (lane & 1) return;
    }
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        const int wi = CH * lane / PW + k;   // 32-bit word of the token
        *reinterpret_cast<uint32_t *>(rec + ((wi >> 2) * kLatTok + t) * 16 + (wi & 3) * 4) = w[k];
    }
}

template <int CH, int BITS>
__global__ void __launch_bounds__(32 * kApWarps)
    latent_append_kernel(LatentGeom g, LatentDev dv, const __half *C, const __half *Kr,
                         const __grid_constant__ LatentTokens a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.y, x = blockIdx.x * kApWarps + warp, n = a.n[i], T = a.T[i];
    kivi_after_previous();
    if (n == 0 || T + x >= lat_end(T, n)) return;
    const int tau = T + x;
    const bool is = x < n;   // (else a place without a token)
    const LatMoves mv = lat_moves(T, n, g.R, g.ring * kLatTok, x);
    const size_t src = (size_t)i * a.n_stride + x;
    LatRow<CH> row;
    uint32_t key = 0;
    if (is) {
        row.load(C + src * g.r, lane);
        key = *reinterpret_cast<const uint32_t *>(Kr + src * kLatRope + 2 * lane);
    } else {
        row.zero();
    }
    // token o to codes; in the block of Tq1 the ring keeps it, as they restore it
    auto quantize = [&](int o, LatRow<CH> &r) {
        lat_quantize<CH, BITS>(g, dv.rec + lat_rec(g, i, o / kLatTok), o % kLatTok, r);
        if (lat_restored(T, n, g.R, o)) r.store_block(dv.ring + lat_ring(g, i, o / kLatTok), o % kLatTok, lane);
    };
    auto leave = [&](int o) {   // cached token o leaves the window
        LatRow<CH> old;
        old.load_block(dv.ring + lat_ring(g, i, o / kLatTok), o % kLatTok, lane);
        quantize(o, old);
    };
    if (mv.own >= 0) leave(mv.own);
    if (mv.under >= 0) leave(mv.under);
    if (mv.codes) quantize(tau, row);
    else row.store_block(dv.ring + lat_ring(g, i, tau / kLatTok), tau % kLatTok, lane);
    if (is)
        *reinterpret_cast<uint32_t *>((char *)(dv.kr + lat_kr(g, i, tau / kLatTok)) + lat_at(lane >> 2, tau % kLatTok, kLatTok) +
                                      (lane & 3) * 4) = key;
}

// The cache as attention sees it, and new tokens behind it: 8 channels a thread.
__global__ void latent_rows_kernel(LatentGeom g, LatentDev dv, const __half *Cn, const __half *Krn, __half *C, __half *Kr, int stride,
                                   const __grid_constant__ LatentTokens a) {
    const int i = blockIdx.y, per = (g.r + kLatRope) / 8;
    const long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int tau = (int)(e / per), c = (int)(e % per);
    const int T = a.T[i];
    kivi_after_previous();
    if (tau >= T + a.n[i]) return;
    const int kb = tau / kLatTok, t = tau % kLatTok;
    const size_t row = (size_t)i * stride + tau;
    if (tau >= T) {
        const size_t src = (size_t)i * a.n_stride + (tau - T);
        if (c >= g.r / 8) {
            const int k = c - g.r / 8;
            if (Kr) *reinterpret_cast<uint4 *>(Kr + row * kLatRope + 8 * k) = *reinterpret_cast<const uint4 *>(Krn + src * kLatRope + 8 * k);
        } else if (C) {
            *reinterpret_cast<uint4 *>(C + row * g.r + 8 * c) = *reinterpret_cast<const uint4 *>(Cn + src * g.r + 8 * c);
        }
        return;
    }
    if (c >= g.r / 8) {
        const int k = c - g.r / 8;
        if (Kr)
            *reinterpret_cast<uint4 *>(Kr + row * kLatRope + 8 * k) =
                *reinterpret_cast<const uint4 *>((const char *)(dv.kr + lat_kr(g, i, kb)) + lat_at(k, t, kLatTok));
        return;
    }
    if (!C) return;
    uint4 v;
    if (tau >= lat_tq(T, g.R)) {
        v = *reinterpret_cast<const uint4 *>((const char *)(dv.ring + lat_ring(g, i, kb)) + lat_at(c, t, kLatTok));
    } else {
        const unsigned char *rec = dv.rec + lat_rec(g, i, kb);
        const __half2 sz = *reinterpret_cast<const __half2 *>(rec + g.off_sz + ((8 * c / g.G) * kLatTok + t) * 4);
        const int PW = 32 / g.bits, wi = 8 * c / PW, f0 = (8 * c % PW) >> 1, m = (1 << g.bits) - 1;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + ((wi >> 2) * kLatTok + t) * 16 + (wi & 3) * 4);
        uint32_t *h = reinterpret_cast<uint32_t *>(&v);
        for (int k = 0; k < 4; ++k) {
            const int lo = (w >> (g.bits * (f0 + k))) & m, hi = (w >> (16 + g.bits * (f0 + k))) & m;
            const __half2 y = __hfma2(__halves2half2(__int2half_rn(lo), __int2half_rn(hi)), __low2half2(sz), __high2half2(sz));
            h[k] = *reinterpret_cast<const uint32_t *>(&y);
        }
    }
    *reinterpret_cast<uint4 *>(C + row * g.r + 8 * c) = v;
}

}  // namespace

cudaError_t kivi_launch_latent_append(const LatentGeom &g, const LatentDev &dv, const __half *C, const __half *Kr,
                                      const LatentTokens &a, cudaStream_t st) {
    int most = 0;   // warps of a sequence
    for (int i = 0; i < g.b; ++i)
        if (a.n[i] > 0) most = std::max(most, lat_end(a.T[i], a.n[i]) - a.T[i]);
    const dim3 grid((unsigned)((most + kApWarps - 1) / kApWarps), (unsigned)g.b);
    const auto kernel = g.r == 512 ? (g.bits == 4 ? latent_append_kernel<16, 4> : latent_append_kernel<16, 2>)
                                   : (g.bits == 4 ? latent_append_kernel<8, 4> : latent_append_kernel<8, 2>);
    return kivi_launch_after(kernel, grid, 32 * kApWarps, 0, st, 1, g, dv, C, Kr, a);
}

cudaError_t kivi_launch_latent_rows(const LatentGeom &g, const LatentDev &dv, const __half *Cn, const __half *Krn,
                                    __half *C, __half *Kr, const LatentTokens &a, int stride, int maxS, cudaStream_t st) {
    const long long items = (long long)maxS * ((g.r + kLatRope) / 8);
    return kivi_launch_after(latent_rows_kernel, dim3((unsigned)((items + 255) / 256), (unsigned)g.b), 256, 0, st, 1, g, dv, Cn,
                             Krn, C, Kr, stride, a);
}

bool kivi_device_info(KiviDeviceInfo *info) {
    constexpr int N = 64;
    static std::mutex mu;
    static KiviDeviceInfo known[N];   // (status null: not asked for yet)
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
    std::lock_guard<std::mutex> lk(mu);
    if (dev < N && known[dev].status) {
        *info = known[dev];
        return true;
    }
    void *p = nullptr;
    info->device = dev;
    if (cudaDeviceGetAttribute(&info->sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaGetSymbolAddress(&p, g_status) != cudaSuccess)
        return false;
    info->status = (unsigned *)p;
    if (dev < N) known[dev] = *info;
    return true;
}

// ---------------------------------------------------------------------------
// The handle and the entry points
// ---------------------------------------------------------------------------
struct kivi_latent {
    bool poisoned;
    int max_tokens, device, num_sms;
    LatentGeom g;
    LatentDev dv;
    float *part;            // the attention's partials, made by the first call that cuts row tiles
    std::vector<int> T;     // host mirror: tokens of each sequence
};

namespace {

std::mutex g_mu;
std::set<void *> g_handles;

kivi_status fail(kivi_status s, const char *fmt, long v = 0) {
    char msg[256];
    snprintf(msg, sizeof msg, fmt, v);
    kivi_set_last_error(msg);
    return s;
}
kivi_status fail_cuda(kivi_latent *c, cudaError_t e, const char *where) {
    if (c) c->poisoned = true;
    char msg[256];
    snprintf(msg, sizeof msg, "%s: %s", where, cudaGetErrorString(e));
    kivi_set_last_error(msg);
    return KIVI_ERR_CUDA;
}

kivi_status check(kivi_latent_t c, bool device) {
    if (!c) return fail(KIVI_ERR_INVALID_ARG, "null latent cache handle");
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_handles.count((void *)c)) return fail(KIVI_ERR_INVALID_ARG, "unknown or destroyed latent cache handle");
    }
    if (c->poisoned) return fail(KIVI_ERR_STATE, "latent cache poisoned by an earlier CUDA error");
    int dev = -1;
    if (device && (cudaGetDevice(&dev) != cudaSuccess || dev != c->device))
        return fail(KIVI_ERR_INVALID_ARG, "the latent cache belongs to device %ld, which is not current", c->device);
    return KIVI_OK;
}
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// n and the tensors of new tokens; *maxn: the most of a sequence
kivi_status check_tokens(int b, const void *C, const void *Kr, const int32_t *n, int n_stride, int *maxn) {
    if (!n || n_stride < 0) return fail(KIVI_ERR_INVALID_ARG, "the counts are null or their stride negative");
    if (n_stride > (1 << 26)) return fail(KIVI_ERR_UNSUPPORTED, "a stride above 2^26 tokens");
    *maxn = 0;
    for (int i = 0; i < b; ++i) {
        if (n[i] < 0 || n[i] > n_stride)
            return fail(KIVI_ERR_INVALID_ARG, "the count of sequence %ld is outside its stride", i);
        *maxn = n[i] > *maxn ? n[i] : *maxn;
    }
    if (*maxn > 0 && (!C || !Kr)) return fail(KIVI_ERR_INVALID_ARG, "a tensor pointer is null");
    if (*maxn > 0 && (!aligned16(C) || !aligned16(Kr)))
        return fail(KIVI_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    return KIVI_OK;
}

void free_latent(kivi_latent *c) {
    void *ps[] = {c->dv.rec, c->dv.ring, c->dv.kr, c->dv.status, c->part};
    for (void *p : ps)
        if (p) cudaFree(p);
}

// kivi_latent_append, and kivi_latent_prefill (anew: every sequence is empty before it)
kivi_status put(kivi_latent *c, const void *C, const void *Kr, const int32_t *n, int n_stride, bool anew, const char *what,
                cudaStream_t st) {
    int maxn = 0;
    kivi_status s = check_tokens(c->g.b, C, Kr, n, n_stride, &maxn);
    if (s != KIVI_OK) return s;
    LatentTokens a;
    a.n_stride = n_stride;
    for (int i = 0; i < c->g.b; ++i) {
        a.T[i] = anew ? 0 : c->T[i];
        a.n[i] = n[i];
        if (n[i] > c->max_tokens - a.T[i]) return fail(KIVI_ERR_CAPACITY, "sequence %ld would exceed max_tokens", i);
    }
    if (maxn > 0) {
        const cudaError_t e =
            kivi_launch_latent_append(c->g, c->dv, (const __half *)C, (const __half *)Kr, a, st);
        if (e != cudaSuccess) return fail_cuda(c, e, what);
    }
    for (int i = 0; i < c->g.b; ++i) c->T[i] = a.T[i] + n[i];
    return KIVI_OK;
}

// kivi_latent_restore (n null: every sequence, no new tokens) and kivi_latent_rows
// (sequences with new tokens)
kivi_status rows(kivi_latent *c, const void *Cn, const void *Krn, const int32_t *n, int n_stride, void *C, void *Kr,
                 int stride, const char *what, cudaStream_t st) {
    if (stride < 0) return fail(KIVI_ERR_INVALID_ARG, "the output's stride is negative");
    if ((C && !aligned16(C)) || (Kr && !aligned16(Kr)))
        return fail(KIVI_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    LatentTokens a;
    a.n_stride = n_stride;
    int maxS = 0;
    for (int i = 0; i < c->g.b; ++i) {
        a.n[i] = n ? n[i] : 0;
        a.T[i] = !n || n[i] > 0 ? c->T[i] : 0;
        if (a.n[i] > stride - a.T[i])
            return fail(KIVI_ERR_INVALID_ARG, "sequence %ld has more tokens than the output's stride", i);
        maxS = a.T[i] + a.n[i] > maxS ? a.T[i] + a.n[i] : maxS;
    }
    if (maxS == 0 || (!C && !Kr)) return KIVI_OK;
    const cudaError_t e = kivi_launch_latent_rows(c->g, c->dv, (const __half *)Cn, (const __half *)Krn, (__half *)C,
                                                  (__half *)Kr, a, stride, maxS, st);
    return e == cudaSuccess ? KIVI_OK : fail_cuda(c, e, what);
}

}  // namespace

extern "C" {

kivi_status kivi_latent_create(int b, int r, int bits, int G, int R, int max_tokens, kivi_latent_t *out) {
    kivi_set_last_error("");
    if (!out) return fail(KIVI_ERR_INVALID_ARG, "out is null");
    *out = nullptr;
    if (b < 1 || r < 1 || G < 1 || R < 1 || max_tokens < 1) return fail(KIVI_ERR_INVALID_ARG, "sizes must be positive");
    if (b > KIVI_MAX_BATCH) return fail(KIVI_ERR_UNSUPPORTED, "b above %ld", KIVI_MAX_BATCH);
    if (r != 256 && r != 512) return fail(KIVI_ERR_UNSUPPORTED, "r must be 256 or 512");
    if (bits != 2 && bits != 4) return fail(KIVI_ERR_UNSUPPORTED, "bits must be 2 or 4");
    if (G != 32 && G != 64 && G != 128) return fail(KIVI_ERR_UNSUPPORTED, "G must be 32, 64 or 128");
    if (R % 64 != 0) return fail(KIVI_ERR_UNSUPPORTED, "R must be a multiple of 64");
    if (max_tokens > (1 << 30)) return fail(KIVI_ERR_UNSUPPORTED, "max_tokens above 2^30");
    kivi_latent *c = new (std::nothrow) kivi_latent();
    if (!c) return fail(KIVI_ERR_OOM, "host allocation failed");
    try {
        c->T.assign((size_t)b, 0);
    } catch (...) {
        delete c;
        return fail(KIVI_ERR_OOM, "host allocation failed");
    }
    c->max_tokens = max_tokens;
    LatentGeom &g = c->g;
    g.b = b;
    g.r = r;
    g.bits = bits;
    g.G = G;
    g.blocks = (max_tokens + kLatTok - 1) / kLatTok;
    g.R = R < g.blocks * kLatTok ? R : g.blocks * kLatTok;   // (a window that holds every token)
    g.recs = (lat_tq(max_tokens, g.R) + kLatTok - 1) / kLatTok;
    g.ring = (g.R + kLatTok - 1) / kLatTok + 1;   // (a window's tokens and those before them in their first block)
    g.off_sz = kLatTok * r * bits / 8;
    g.rec_bytes = g.off_sz + r / G * kLatTok * 4;
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device);
    if (e != cudaSuccess) {
        delete c;
        return fail_cuda(nullptr, e, "no CUDA device");
    }
    struct Req { void **p; size_t bytes; } reqs[] = {
        {(void **)&c->dv.rec, (size_t)b * g.recs * g.rec_bytes},
        {(void **)&c->dv.ring, (size_t)b * g.ring * kLatTok * r * 2},
        {(void **)&c->dv.kr, (size_t)b * g.blocks * kLatTok * kLatRope * 2},
        {(void **)&c->dv.status, 4},
    };
    for (auto &q : reqs) {
        if (q.bytes == 0) continue;   // (no records: a window that holds every token)
        e = cudaMalloc(q.p, q.bytes);
        if (e == cudaSuccess) e = cudaMemset(*q.p, 0, q.bytes);
        if (e != cudaSuccess) break;
    }
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        free_latent(c);
        delete c;
        cudaGetLastError();
        fail_cuda(nullptr, e, "device allocation failed");
        return e == cudaErrorMemoryAllocation ? KIVI_ERR_OOM : KIVI_ERR_CUDA;
    }
    try {
        std::lock_guard<std::mutex> lk(g_mu);
        g_handles.insert(c);
    } catch (...) {
        free_latent(c);
        delete c;
        return fail(KIVI_ERR_OOM, "host allocation failed");
    }
    *out = c;
    return KIVI_OK;
}

kivi_status kivi_latent_destroy(kivi_latent_t c) {
    kivi_set_last_error("");
    if (!c) return fail(KIVI_ERR_INVALID_ARG, "null latent cache handle");
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_handles.erase((void *)c)) return fail(KIVI_ERR_INVALID_ARG, "unknown or destroyed latent cache handle");
    }
    cudaDeviceSynchronize();
    cudaGetLastError();
    free_latent(c);
    delete c;
    return KIVI_OK;
}

kivi_status kivi_latent_prefill(kivi_latent_t c, const void *C, const void *Kr, const int32_t *t, int t_stride,
                                kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    return put(c, C, Kr, t, t_stride, true, "latent_prefill", (cudaStream_t)stream);
}

kivi_status kivi_latent_append(kivi_latent_t c, const void *C, const void *Kr, const int32_t *n, int n_stride,
                               kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    return put(c, C, Kr, n, n_stride, false, "latent_append", (cudaStream_t)stream);
}

kivi_status kivi_latent_attn(kivi_latent_t c, const void *q, const void *q_rope, const void *C, const void *Kr,
                             const int32_t *n, int n_stride, int h, float scale, void *out, kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    if (h < 1) return fail(KIVI_ERR_INVALID_ARG, "h must be positive");
    if (h > 128) return fail(KIVI_ERR_UNSUPPORTED, "more than 128 heads");
    if (!(scale > 0.f && scale - scale == 0.f)) return fail(KIVI_ERR_INVALID_ARG, "scale must be positive and finite");
    int maxn = 0;
    s = check_tokens(c->g.b, C, Kr, n, n_stride, &maxn);
    if (s != KIVI_OK) return s;
    if (maxn == 0) return KIVI_OK;
    if (!q || !q_rope || !out) return fail(KIVI_ERR_INVALID_ARG, "q, q_rope or out is null");
    if (!aligned16(q) || !aligned16(q_rope) || !aligned16(out))
        return fail(KIVI_ERR_INVALID_ARG, "q, q_rope and out must be 16-byte aligned");
    if ((long long)c->g.b * n_stride >= (1LL << 31)) return fail(KIVI_ERR_UNSUPPORTED, "b n_stride must be below 2^31");
    if ((long long)n_stride * h >= (1LL << 24)) return fail(KIVI_ERR_UNSUPPORTED, "n_stride h must be below 2^24");
    ChunkArgs a;
    for (int i = 0; i < c->g.b; ++i) {
        a.T[i] = c->T[i];
        a.Tqk[i] = a.Tqv[i] = lat_tq(c->T[i], c->g.R);
        a.n[i] = n[i];
    }
    a.n_stride = n_stride;
    ChunkPlan plan;
    if (!kivi_plan_latent(c->g, h, a, c->num_sms, &plan))
        return fail(KIVI_ERR_UNSUPPORTED, "more than 2^31 key tiles an SM");
    if (plan.join && !c->part) {
        // (relaxed: the allocation is legal, and not part of the graph, while a stream is captured)
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        cudaThreadExchangeStreamCaptureMode(&mode);
        const cudaError_t e = cudaMalloc((void **)&c->part, kivi_latent_partial_floats(c->g, c->num_sms) * 4);
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess) {
            c->part = nullptr;
            if (e != cudaErrorMemoryAllocation) return fail_cuda(c, e, "partials");
            cudaGetLastError();
            return fail(KIVI_ERR_OOM, "no device memory for the partials");
        }
    }
    const cudaError_t e = kivi_launch_latent_attn(c->g, c->dv, (const __half *)q, (const __half *)q_rope,
                                                  (const __half *)C, (const __half *)Kr, (__half *)out, a, plan, scale,
                                                  c->part, c->device, c->num_sms, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(c, e, "latent_attn");
    return KIVI_OK;
}

kivi_status kivi_latent_lengths(kivi_latent_t c, int32_t *T, int32_t *Tq) {
    kivi_set_last_error("");
    kivi_status s = check(c, false);
    if (s != KIVI_OK && s != KIVI_ERR_STATE) return s;
    for (int i = 0; i < c->g.b; ++i) {
        if (T) T[i] = c->T[i];
        if (Tq) Tq[i] = lat_tq(c->T[i], c->g.R);
    }
    return KIVI_OK;
}

kivi_status kivi_latent_restore(kivi_latent_t c, void *C, void *Kr, int t_stride, kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    return rows(c, nullptr, nullptr, nullptr, 0, C, Kr, t_stride, "latent_restore", (cudaStream_t)stream);
}

kivi_status kivi_latent_rows(kivi_latent_t c, const void *C, const void *Kr, const int32_t *n, int n_stride, void *C_out,
                             void *Kr_out, int s_stride, kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    int maxn = 0;
    s = check_tokens(c->g.b, C, Kr, n, n_stride, &maxn);
    if (s != KIVI_OK) return s;
    return maxn == 0 ? KIVI_OK : rows(c, C, Kr, n, n_stride, C_out, Kr_out, s_stride, "latent_rows", (cudaStream_t)stream);
}

kivi_status kivi_latent_product(kivi_latent_t c, const void *x, const void *w, int h_x, int h, int n_stride,
                                const int32_t *n, int K, int N, int transposed, void *out, kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    s = kivi_head_product_to(c->dv.status, x, w, c->g.b, h_x, h, n_stride, n, K, N, transposed, out, stream);
    c->poisoned |= s == KIVI_ERR_CUDA;
    return s;
}

kivi_status kivi_latent_expanded(kivi_latent_t c, const void *q, const void *q_rope, const void *K, const void *Kr,
                                 const void *V, int h, const int32_t *T, const int32_t *n, int n_stride, int s_stride,
                                 float scale, void *out, kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    s = kivi_latent_expanded_to(c->dv.status, q, q_rope, K, Kr, V, c->g.b, h, T, n, n_stride, s_stride, scale, out, stream);
    c->poisoned |= s == KIVI_ERR_CUDA;
    return s;
}

kivi_status kivi_latent_check(kivi_latent_t c, uint32_t *flags, kivi_stream_t stream) {
    kivi_set_last_error("");
    kivi_status s = check(c, true);
    if (s != KIVI_OK) return s;
    if (!flags) return fail(KIVI_ERR_INVALID_ARG, "flags is null");
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaMemcpyAsync(flags, c->dv.status, 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) e = cudaMemsetAsync(c->dv.status, 0, 4, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return fail_cuda(c, e, "latent_check");
    return KIVI_OK;
}

kivi_status kivi_device_check(uint32_t *flags, kivi_stream_t stream) {
    kivi_set_last_error("");
    if (!flags) return fail(KIVI_ERR_INVALID_ARG, "flags is null");
    KiviDeviceInfo info;
    if (!kivi_device_info(&info)) return fail(KIVI_ERR_CUDA, "no status word on the current device");
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaMemcpyAsync(flags, info.status, 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) e = cudaMemsetAsync(info.status, 0, 4, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e == cudaSuccess ? KIVI_OK : fail_cuda(nullptr, e, "device_check");
}

}  // extern "C"
