// kivi_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers, and the entry point kivi_verify.
//
// Mathematics.  Drafted token x_r of a sequence was drawn from q_r; the
// target's probabilities at its place are p_r.  Token r is kept while
// u_r q_r(x_r) < p_r(x_r); at the first that is not, one token is drawn from
// the weights max(p_r - q_r, 0), after a whole draft from p_n: the tokens are
// then distributed as the target's.  (The products u q are exact in 64 bits.)
//
// The drawing is in whole numbers: a probability counts floor(2^40 p) units,
// weights are their differences and W their sum, below 2^60.  The token is the
// lowest i whose weights up to and with it exceed floor(U W / 2^30), U =
// floor(2^30 u).  Sums of whole numbers do not depend on their order, so the
// split over threads and CTAs does not show in the result.
//
// Bound: latency, for all that two rows of the vocabulary a sequence have to come from
// memory: draft -> its probabilities -> the row, 8 values a lane at a time, each time
// waiting for the last (64 x 32000: 2, 16 x 150001: 5) -> the cluster's sums -> the
// stretch again.  A
// cluster of CTAs shares a sequence: each warp sums a stretch of the row (the
// units are never stored), the CTAs exchange their warps' sums through
// distributed shared memory, and the CTA whose stretch holds the mark reads
// that warp's stretch again, a few values a thread.
#include <cooperative_groups.h>

#include "../../include/kivi.h"
#include "kivi_latent.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kVfThreads = 512, kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCluster = 8;
constexpr int kVfUnroll = 8;   // values of a row in flight a thread

typedef unsigned long long u64;

struct VerifyArgs {
    const void *p, *q;      // [b][n_stride + 1][V], [b][n_stride][V] (or null: the draft is certain)
    const int *draft;       // [b][n_stride]
    const float *u;         // [b][n_stride + 1]
    int *tokens, *accepted; // [b][n_stride + 1], [b]
    int n_stride, V;
    int per;                // values a warp sums (a multiple of 32)
    int n[KIVI_MAX_BATCH];
};

__device__ __forceinline__ float vf_float(float x) { return x; }
__device__ __forceinline__ float vf_float(__half x) { return __half2float(x); }
// units of a probability: its 24 bits, shifted (conversions to 64-bit integers
// are slow here); not a number and below zero: none, above one: one
__device__ __forceinline__ u64 vf_units(float p) {
    const unsigned b = p > 0.f ? min(__float_as_uint(p), 0x3f800000u) : 0u;
    const int d = (int)(b >> 23) - 110;   // 2^40 p = m 2^d
    const unsigned m = ((b & 0x7fffffu) | 0x800000u) >> min(max(-d, 0), 31);
    return (u64)m << max(d, 0);
}
__device__ __forceinline__ u64 vf_warp_sum(u64 x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a sequence draws from: row p, less row q (or one unit row at `one`)
// where the token there was not kept.
template <typename T>
struct VfRow {
    const T *p, *q;   // q null: nothing is taken off, but at `one`
    int one;          // -1: none
    __device__ __forceinline__ u64 weight(int i, u64 units, float qi) const {
        const u64 off = q ? vf_units(qi) : i == one ? 1ull << 40 : 0ull;
        return units > off ? units - off : 0ull;
    }
};

// Grid (cluster, b).
template <typename T>
__global__ void __launch_bounds__(kVfThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    __shared__ u64 s_sum[2][kVfMaxCluster][kVfWarps];   // the warps' weights, and units of p, of every CTA
    __shared__ u64 s_scan[kVfWarps];
    __shared__ u64 s_mark, s_before;
    __shared__ int s_first, s_which;
    __shared__ bool s_plain;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i = blockIdx.y, rank = blockIdx.x, C = gridDim.x, n = a.n[i];
    const T *P = (const T *)a.p + (size_t)i * (a.n_stride + 1) * a.V;
    const T *Q = a.q ? (const T *)a.q + (size_t)i * a.n_stride * a.V : nullptr;
    const int *draft = a.draft + (size_t)i * a.n_stride;
    const float *u = a.u + (size_t)i * (a.n_stride + 1);

    const float uu = u[a.n_stride];
    cl.barrier_arrive();   // (waited for before the first store to another CTA: it has started)
    // the first token that is not kept (every CTA finds it for itself)
    if (warp == 0) {
        int first = n;
        for (int r0 = 0; r0 < n; r0 += 32) {
            const int r = r0 + lane;
            bool drop = false;
            if (r < n) {
                const int x = draft[r];
                const bool in = (unsigned)x < (unsigned)a.V;   // a token outside the vocabulary is not kept
                const float px = in ? vf_float(P[(size_t)r * a.V + x]) : 0.f;
                const float qx = in && Q ? vf_float(Q[(size_t)r * a.V + x]) : 1.f;
                drop = !((double)u[r] * (double)qx < (double)px);
            }
            const unsigned m = __ballot_sync(0xffffffffu, drop);
            if (m) {
                first = r0 + __ffs(m) - 1;
                break;
            }
        }
        if (lane == 0) s_first = first;
    }
    __syncthreads();
    const int first = s_first;
    VfRow<T> row;
    row.p = P + (size_t)first * a.V;
    row.q = first < n && Q ? Q + (size_t)first * a.V : nullptr;
    row.one = first < n && !Q ? draft[first] : -1;

    // each warp's sums over its stretch
    const int lo = min((rank * kVfWarps + warp) * a.per, a.V), hi = min(lo + a.per, a.V);
    u64 sw = 0, sp = 0;
    for (int e0 = lo + lane; e0 < hi; e0 += 32 * kVfUnroll) {
        T x[kVfUnroll], y[kVfUnroll];
#pragma unroll
        for (int k = 0; k < kVfUnroll; ++k) {
            const int e = min(e0 + 32 * k, hi - 1);
            x[k] = row.p[e];
            if (row.q) y[k] = row.q[e];
        }
#pragma unroll
        for (int k = 0; k < kVfUnroll; ++k) {
            if (e0 + 32 * k >= hi) break;
            const u64 un = vf_units(vf_float(x[k]));
            sp += un;
            sw += row.weight(e0 + 32 * k, un, row.q ? vf_float(y[k]) : 0.f);
        }
    }
    sw = vf_warp_sum(sw);
    sp = vf_warp_sum(sp);
    cl.barrier_wait();
    // to every CTA (then none reads another's shared memory, which may be given up)
    if (lane < C) {
        u64 *s = cl.map_shared_rank(&s_sum[0][rank][warp], lane);
        s[0] = sw;
        s[kVfMaxCluster * kVfWarps] = sp;
    }
    cl.sync();
    // the stretch that holds the mark (every CTA finds it for itself: the first warp,
    // the sums of all CTAs' warps lane by lane)
    if (warp == 0) {
        constexpr int NK = kVfMaxCluster * kVfWarps / 32;
        const u64 *sums = &s_sum[0][0][0];
        u64 w[NK], tw = 0;
        auto take = [&]() {
            tw = 0;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                w[k] = 32 * k + lane < C * kVfWarps ? sums[32 * k + lane] : 0ull;
                tw += w[k];
            }
            tw = vf_warp_sum(tw);
        };
        take();
        const bool plain = tw == 0;   // nothing left of the difference: p itself
        if (plain) {
            sums += kVfMaxCluster * kVfWarps;
            take();
        }
        // floor(U W / 2^30)
        const u64 U = uu > 0.f ? __float2uint_rz(fminf(uu, 1.f - 0x1p-24f) * 0x1p30f) : 0u;
        const u64 mark = U * (tw >> 30) + ((U * (tw & ((1ull << 30) - 1))) >> 30);
        u64 before = 0;
        int which = -1;   // (none: no weight at all)
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            if (32 * k >= C * kVfWarps || which >= 0 || tw == 0) break;
            u64 c = w[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += v;
            }
            const unsigned m = __ballot_sync(0xffffffffu, before + c > mark);
            if (m) {
                which = 32 * k + __ffs(m) - 1;
                before += __shfl_sync(0xffffffffu, c - w[k], __ffs(m) - 1);
            } else {
                before += __shfl_sync(0xffffffffu, c, 31);
            }
        }
        if (lane == 0) {
            s_mark = mark;
            s_before = before;
            s_which = which;
            s_plain = plain;
        }
    }
    __syncthreads();
    const int which = s_which;
    if (rank == 0) {
        for (int r = tid; r <= a.n_stride; r += kVfThreads)
            if (r != first || which < 0) a.tokens[(size_t)i * (a.n_stride + 1) + r] = r < first ? draft[r] : -1;
        if (tid == 0) a.accepted[i] = first;
    }
    if (which < 0 || which / kVfWarps != rank) return;
    const u64 mark = s_mark, before = s_before;
    const bool plain = s_plain;
    // this CTA's threads share that stretch
    const int l0 = which * a.per, l1 = min(l0 + a.per, a.V), share = (l1 - l0 + kVfThreads - 1) / kVfThreads;
    const int t0 = min(l0 + tid * share, l1), t1 = min(t0 + share, l1);
    auto at = [&](int e) {
        const u64 un = vf_units(vf_float(row.p[e]));
        return plain ? un : row.weight(e, un, row.q ? vf_float(row.q[e]) : 0.f);
    };
    u64 mine = 0;
    for (int e = t0; e < t1; ++e) mine += at(e);
    u64 c = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += v;
    }
    if (lane == 31) s_scan[warp] = c;
    __syncthreads();
    u64 base = before + c - mine;
    for (int k = 0; k < warp; ++k) base += s_scan[k];
    if (base <= mark && mark < base + mine) {
        int e = t0;
        for (u64 x = base; e < t1; ++e) {
            x += at(e);
            if (x > mark) break;
        }
        a.tokens[(size_t)i * (a.n_stride + 1) + first] = e;
    }
}

kivi_status fail(kivi_status s, const char *msg) {
    kivi_set_last_error(msg);
    return s;
}

}  // namespace

extern "C" kivi_status kivi_verify(const void *p, const void *q, int bytes, const int32_t *draft, const float *u, int b,
                                   int n_stride, int vocab, const int32_t *n, int32_t *tokens, int32_t *accepted,
                                   kivi_stream_t stream) {
    kivi_set_last_error("");
    if (b < 1 || n_stride < 0 || vocab < 1) return fail(KIVI_ERR_INVALID_ARG, "sizes must be positive");
    if (b > KIVI_MAX_BATCH) return fail(KIVI_ERR_UNSUPPORTED, "b above 1024");
    if (vocab > (1 << 20)) return fail(KIVI_ERR_UNSUPPORTED, "a vocabulary above 2^20");
    if (n_stride > (1 << 20)) return fail(KIVI_ERR_UNSUPPORTED, "n_stride above 2^20");
    if (bytes != 2 && bytes != 4) return fail(KIVI_ERR_UNSUPPORTED, "probabilities have 2 or 4 bytes");
    if (!n || !p || !u || !tokens || !accepted || (n_stride > 0 && !draft))
        return fail(KIVI_ERR_INVALID_ARG, "a pointer is null");
    if (((uintptr_t)p | (uintptr_t)q) & (unsigned)(bytes - 1))
        return fail(KIVI_ERR_INVALID_ARG, "p and q must be aligned to their values");
    if (((uintptr_t)draft | (uintptr_t)u | (uintptr_t)tokens | (uintptr_t)accepted) & 3u)
        return fail(KIVI_ERR_INVALID_ARG, "draft, u, tokens and accepted must be 4-byte aligned");
    VerifyArgs A;
    for (int i = 0; i < b; ++i) {
        if (n[i] < 0 || n[i] > n_stride) return fail(KIVI_ERR_INVALID_ARG, "n[i] outside [0, n_stride]");
        A.n[i] = n[i];
    }
    A.p = p;
    A.q = q;
    A.draft = draft;
    A.u = u;
    A.tokens = tokens;
    A.accepted = accepted;
    A.n_stride = n_stride;
    A.V = vocab;
    // CTAs a sequence: eight (with sixteen, 16 sequences of 150001 took 15.2 us for
    // 14.0), fewer where the vocabulary is small, or where they would not all run at
    // once, two an SM (64 sequences of 32000: 11.1 us with eight and two waves, 10.2)
    KiviDeviceInfo info;
    if (!kivi_device_info(&info)) return fail(KIVI_ERR_CUDA, "no current device");
    int C = kVfMaxCluster;
    while (C > 1 && (vocab < 2048 * C || (long long)b * C > 2 * info.sms)) C >>= 1;
    A.per = (vocab + C * kVfWarps - 1) / (C * kVfWarps);
    A.per = (A.per + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, (unsigned)b);
    cfg.blockDim = dim3(kVfThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaError_t e = bytes == 4 ? cudaLaunchKernelEx(&cfg, verify_kernel<float>, A)
                               : cudaLaunchKernelEx(&cfg, verify_kernel<__half>, A);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? KIVI_OK : fail(KIVI_ERR_CUDA, cudaGetErrorString(e));
}
