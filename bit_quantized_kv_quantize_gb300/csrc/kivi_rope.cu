// kivi_rope.cu -- rotary positions of queries and keys, and the entry points
// kivi_rope and kivi_rope_axes.
//
// Mathematics.  Channel pair m of a token at position p turns by the angle
// p w_m:  (x, y) -> f (x cos - y sin, y cos + x sin), with w_m the pair's
// frequency and f one factor for the whole rotated part.  Pairs are
// channels (m, m + rot/2) (half layout) or (2m, 2m + 1) (interleaved);
// channels past rot stay as they are.
//
// Angles.  At position 10^6 a 32-bit product p w_m is off by a large part
// of a radian, and 64-bit floating point is slow on this GPU.  So a
// frequency is held as a fixed-point fraction of a full turn, 2^64 = one
// turn: the 64-bit integer product with the position drops the whole turns
// by itself (negative positions too), is exact up to the frequency's own
// rounding (2^-65 turn a position), and its top 32 bits, read as a signed
// number, are the angle in half turns for sincospi.
//
// Several axes (a patch's time, height and width): pair m turns by the token's
// position on axis[m].  A thread of one axis loads one position, of several
// eight (from the first-level cache, all in flight at once); the rest is the
// same.
//
// Bound: memory (4 bytes a value moved, 1.5 multiply-adds a value).  A
// thread keeps the sines and cosines of one token's 8 pairs in registers
// (computing them costs as much as rotating about 6 heads) and applies them
// to several heads, two 16-byte loads and stores a head, four heads in
// flight: 4 x 8192 tokens of 40 heads 99 us (671 MB, 98.9 us at the copy
// rate).  With few tokens, heads are spread over threads instead, one a
// thread: a decode step of 64 sequences, bound by one round trip to memory,
// takes 2.3 us.
#include "../../include/kivi.h"
#include "kivi_internal.cuh"

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;   // d <= 256

struct RopeArgs {
    const __half *src[2];   // q, k (null: absent)
    __half *dst[2];
    int heads[2];
    int n_stride, rot;
    float factor;
    bool inverse;
    const int *pos;         // device positions [axes][b][n_stride], or null: pos0[i] + r
    int n[KIVI_MAX_BATCH], pos0[KIVI_MAX_BATCH];
    unsigned long long turns[kRopeMaxPairs];
    uint8_t axis[kRopeMaxPairs];   // (with several axes)
};

__device__ __forceinline__ uint32_t rot_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One block: TR tokens x D / 16 units of 16 channels x HY heads; a thread
// takes heads hy, hy + HY gridDim.y, ... of its unit (q's heads first).
template <int D, bool INTER, bool AXES>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeArgs A, int lgTR, int lgHY) {
    constexpr int U = D / 16;
    const int u = threadIdx.x % U, tr = (threadIdx.x / U) & ((1 << lgTR) - 1), hy = (threadIdx.x / U) >> lgTR;
    const int i = blockIdx.z, r = (blockIdx.x << lgTR) + tr;
    if (r >= A.n[i]) return;
    const bool turn = 16 * u < A.rot;   // else: two chunks that stay as they are
    const int c0 = turn ? (INTER ? 16 * u : 8 * u) : 16 * u;
    const int c1 = turn && !INTER ? A.rot / 2 + 8 * u : c0 + 8;
    float cs[8], sn[8];
    if (turn) {
        long long p[8];
        if (AXES) {
            const size_t plane = (size_t)gridDim.z * A.n_stride;   // (a block of z a sequence)
            const int *pos = A.pos + (size_t)i * A.n_stride + r;
#pragma unroll
            for (int m = 0; m < 8; ++m) p[m] = pos[A.axis[8 * u + m] * plane];
        } else {
            p[0] = A.pos ? A.pos[(size_t)i * A.n_stride + r] : (long long)A.pos0[i] + r;
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const unsigned long long a = (unsigned long long)p[AXES ? m : 0] * A.turns[8 * u + m];
            sincospif((float)(int)(a >> 32) * 0x1p-31f, &sn[m], &cs[m]);
            cs[m] *= A.factor;
            sn[m] *= A.inverse ? -A.factor : A.factor;
        }
    }
    const int H = A.heads[0] + A.heads[1];
    const int step = gridDim.y << lgHY;
    auto row = [&](int h, bool dst) {
        const int w = h < A.heads[0] ? 0 : 1;
        const size_t o = (((size_t)i * A.heads[w] + (w ? h - A.heads[0] : h)) * A.n_stride + r) * D;
        return dst ? A.dst[w] + o : const_cast<__half *>(A.src[w]) + o;
    };
    for (int h0 = (blockIdx.y << lgHY) + hy; h0 < H; h0 += 4 * step) {
        uint4 x[4], y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + k * step;
            if (h >= H) break;
            const __half *s = row(h, false);
            x[k] = *reinterpret_cast<const uint4 *>(s + c0);
            y[k] = *reinterpret_cast<const uint4 *>(s + c1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + k * step;
            if (h >= H) break;
            if (turn) {
                uint32_t *px = reinterpret_cast<uint32_t *>(&x[k]), *py = reinterpret_cast<uint32_t *>(&y[k]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&px[e]));
                    const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&py[e]));
                    if (INTER) {   // pairs e (of x) and 4 + e (of y)
                        px[e] = rot_pair(a.x * cs[e] - a.y * sn[e], a.y * cs[e] + a.x * sn[e]);
                        py[e] = rot_pair(b.x * cs[4 + e] - b.y * sn[4 + e], b.y * cs[4 + e] + b.x * sn[4 + e]);
                    } else {       // pairs 2e and 2e + 1, x with y
                        px[e] = rot_pair(a.x * cs[2 * e] - b.x * sn[2 * e], a.y * cs[2 * e + 1] - b.y * sn[2 * e + 1]);
                        py[e] = rot_pair(b.x * cs[2 * e] + a.x * sn[2 * e], b.y * cs[2 * e + 1] + a.y * sn[2 * e + 1]);
                    }
                }
            }
            __half *t = row(h, true);
            *reinterpret_cast<uint4 *>(t + c0) = x[k];
            *reinterpret_cast<uint4 *>(t + c1) = y[k];
        }
    }
}

template <int D>
cudaError_t launch_rope(const RopeArgs &A, int b, bool interleaved, bool axes, int maxn, cudaStream_t st) {
    constexpr int U = D / 16;
    int lgTR = 0;   // tokens a block: as many as there are, up to the block's threads
    while ((1 << lgTR) < maxn && (U << lgTR) < kRopeThreads) ++lgTR;
    int lgHY = 0;
    while ((U << (lgTR + lgHY)) < kRopeThreads) ++lgHY;
    const int H = A.heads[0] + A.heads[1];
    const unsigned gx = ((unsigned)maxn + (1u << lgTR) - 1) >> lgTR;
    const int rows = (H + (1 << lgHY) - 1) >> lgHY;   // heads a thread would take alone
    // heads a thread: eight (each thread forms the sines of its token once),
    // fewer while that leaves half of the SMs without a block.  40 heads, eight
    // a thread and one, in microseconds: 4 x 8192 tokens 99 and 238, 2048
    // tokens 8.1 and 16.6, 512 tokens 4.3 and 5.8, 64 tokens 4.2 and 2.4.
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int per = 8;
    while (per > 1 && (long long)gx * b * ((rows + per - 1) / per) < sms / 2) per >>= 1;
    const dim3 grid(gx, (rows + per - 1) / per, b);
    if (interleaved && axes) rope_kernel<D, true, true><<<grid, kRopeThreads, 0, st>>>(A, lgTR, lgHY);
    else if (interleaved) rope_kernel<D, true, false><<<grid, kRopeThreads, 0, st>>>(A, lgTR, lgHY);
    else if (axes) rope_kernel<D, false, true><<<grid, kRopeThreads, 0, st>>>(A, lgTR, lgHY);
    else rope_kernel<D, false, false><<<grid, kRopeThreads, 0, st>>>(A, lgTR, lgHY);
    return cudaGetLastError();
}

kivi_status fail(kivi_status s, const char *msg) {
    kivi_set_last_error(msg);
    return s;
}

// kivi_rope, and with axes > 0 kivi_rope_axes (pos then has axes planes)
kivi_status rope(const void *q, const void *k, int b, int h_q, int h_kv, int n_stride, int d, const int32_t *n,
                 const int32_t *pos0, const int32_t *pos, int axes, const uint8_t *axis, const uint64_t *turns,
                 int rot_dim, int interleaved, float factor, int inverse, void *q_out, void *k_out,
                 kivi_stream_t stream) {
    if (b < 1 || n_stride < 0 || h_q < 0 || h_kv < 0 || h_q + (long long)h_kv < 1)
        return fail(KIVI_ERR_INVALID_ARG, "sizes must be positive");
    if (b > KIVI_MAX_BATCH) return fail(KIVI_ERR_UNSUPPORTED, "b above 1024");
    if (d != 64 && d != 128 && d != 256) return fail(KIVI_ERR_UNSUPPORTED, "d must be 64, 128 or 256");
    if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0)
        return fail(KIVI_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16, at most d");
    if (h_q > 65536 || h_kv > 65536) return fail(KIVI_ERR_UNSUPPORTED, "more than 65536 heads");
    if (!n || !turns || (pos0 != nullptr) == (pos != nullptr))
        return fail(KIVI_ERR_INVALID_ARG, axes > 0 ? "need n, turns and pos" : "need n, turns and one of pos0 and pos");
    if (!(factor - factor == 0.f)) return fail(KIVI_ERR_INVALID_ARG, "factor must be finite");
    if ((uintptr_t)pos & 3u) return fail(KIVI_ERR_INVALID_ARG, "pos must be 4-byte aligned");
    RopeArgs A;
    for (int m = 0; axes > 0 && m < kRopeMaxPairs; ++m) {
        A.axis[m] = m < rot_dim / 2 ? axis[m] : 0;
        if (A.axis[m] >= axes) return fail(KIVI_ERR_INVALID_ARG, "a pair's axis is outside [0, axes)");
    }
    int maxn = 0;
    for (int i = 0; i < b; ++i) {
        if (n[i] < 0 || n[i] > n_stride) return fail(KIVI_ERR_INVALID_ARG, "n[i] outside [0, n_stride]");
        A.n[i] = n[i];
        A.pos0[i] = pos0 ? pos0[i] : 0;
        maxn = n[i] > maxn ? n[i] : maxn;
    }
    if (maxn == 0) return KIVI_OK;
    const void *in[2] = {q, k};
    void *out[2] = {q_out, k_out};
    const int heads[2] = {h_q, h_kv};
    for (int w = 0; w < 2; ++w) {
        if (heads[w] > 0 && (!in[w] || !out[w])) return fail(KIVI_ERR_INVALID_ARG, "a tensor pointer is null");
        if (heads[w] > 0 && (((uintptr_t)in[w] | (uintptr_t)out[w]) & 15u))
            return fail(KIVI_ERR_INVALID_ARG, "q, k and the outputs must be 16-byte aligned");
        A.src[w] = (const __half *)in[w];
        A.dst[w] = (__half *)out[w];
        A.heads[w] = heads[w];
    }
    A.n_stride = n_stride;
    A.rot = rot_dim;
    A.factor = factor;
    A.inverse = inverse != 0;
    A.pos = pos;
    for (int m = 0; m < kRopeMaxPairs; ++m) A.turns[m] = m < rot_dim / 2 ? turns[m] : 0ull;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool il = interleaved != 0, ax = axes > 0;
    const cudaError_t e = d == 64 ? launch_rope<64>(A, b, il, ax, maxn, st)
                                  : d == 128 ? launch_rope<128>(A, b, il, ax, maxn, st)
                                             : launch_rope<256>(A, b, il, ax, maxn, st);
    return e == cudaSuccess ? KIVI_OK : fail(KIVI_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace

extern "C" kivi_status kivi_rope(const void *q, const void *k, int b, int h_q, int h_kv, int n_stride, int d,
                                 const int32_t *n, const int32_t *pos0, const int32_t *pos, const uint64_t *turns,
                                 int rot_dim, int interleaved, float factor, int inverse, void *q_out, void *k_out,
                                 kivi_stream_t stream) {
    kivi_set_last_error("");
    return rope(q, k, b, h_q, h_kv, n_stride, d, n, pos0, pos, 0, nullptr, turns, rot_dim, interleaved, factor,
                inverse, q_out, k_out, stream);
}

extern "C" kivi_status kivi_rope_axes(const void *q, const void *k, int b, int h_q, int h_kv, int n_stride, int d,
                                      const int32_t *n, const int32_t *pos, int axes, const uint8_t *axis,
                                      const uint64_t *turns, int rot_dim, int interleaved, float factor, int inverse,
                                      void *q_out, void *k_out, kivi_stream_t stream) {
    kivi_set_last_error("");
    if (axes < 1 || axes > 255) return fail(KIVI_ERR_INVALID_ARG, "axes outside [1, 255]");
    if (!axis) return fail(KIVI_ERR_INVALID_ARG, "axis is null");
    return rope(q, k, b, h_q, h_kv, n_stride, d, n, nullptr, pos, axes, axis, turns, rot_dim, interleaved, factor,
                inverse, q_out, k_out, stream);
}
