// kivi_latent.cuh -- what the host and the kernels of the latent cache share:
// its geometry and layout, and the launchers.
//
// Per sequence the cache holds each token's latent vector c [r] and rotary key
// kr [64].  Tokens [0, Tq) are quantized, a token's groups of G channels with an
// fp16 scale and zero each (the value side of the KIVI quantizer); the newest
// R, [Tq, T), are fp16.  Device memory, tokens in blocks of 128 (an attention
// tile):
//   records  [b][blocks that codes can reach]: codes, then scales and zeros.
//            16-byte words of codes [r bits / 128][128 tokens]: word x of a token
//            covers channels (128 / bits) x ..  In each 32-bit word (16-bit half h,
//            field f of `bits` bits) is the code of channel 2 f + h of the word's 32 /
//            bits.  Scale and zero, a half2, [r / G][128 tokens].
//   ring     [b][ring blocks] and rotary keys [b][blocks]: fp16 blocks as an
//            attention tile holds them (lat_at), so that a block is copied into
//            one as it is.  Token tau of the window is in the ring's block
//            (tau / 128) mod (ring blocks).  The block of Tq holds its quantized
//            tokens too, as their codes restore them: every block from Tq / 128 on
//            is there whole, the places behind the last token zero.
#pragma once
#include <atomic>

#include "../../include/kivi.h"
#include "kivi_chunk.cuh"
#include "kivi_internal.cuh"
#include "kivi_latent_places.h"

constexpr int kLatRope = 64;    // channels of the rotary key
constexpr int kLatHead = 128;   // channels of a head's other keys, and of its values

struct LatentGeom {
    int b, r, bits, G, R;
    int blocks;      // of a sequence
    int recs;        // its records: blocks up to the last that can hold a quantized token
    int ring;        // blocks of its ring
    int off_sz;      // scales and zeros in a record (bytes)
    int rec_bytes;
};
struct LatentDev {
    unsigned char *rec;
    __half *ring, *kr;
    unsigned *status;
};

__host__ __device__ __forceinline__ size_t lat_rec(const LatentGeom &g, int i, int kb) {
    return ((size_t)i * g.recs + kb) * g.rec_bytes;
}
// a block of the ring, of the rotary keys (halves)
__host__ __device__ __forceinline__ size_t lat_ring(const LatentGeom &g, int i, int kb) {
    return ((size_t)i * g.ring + kb % g.ring) * kLatTok * g.r;
}
__host__ __device__ __forceinline__ size_t lat_kr(const LatentGeom &g, int i, int kb) {
    return ((size_t)i * g.blocks + kb) * kLatTok * kLatRope;
}
// Byte of 16-byte chunk c (8 channels) of row t of a block: 64 channels of every
// row together, a row 128 bytes, its chunks in the 128-byte swizzle (which the
// tensor cores read along either axis at their full rate).
__host__ __device__ __forceinline__ unsigned lat_at(int c, int t, int rows) {
    return (unsigned)((c >> 3) * rows * 128 + t * 128 + (((c ^ t) & 7) << 4));
}

// n[i] tokens at positions T[i].. (counts from the host mirror)
struct LatentTokens {
    int n_stride;
    int T[KIVI_MAX_BATCH], n[KIVI_MAX_BATCH];
};

cudaError_t kivi_launch_latent_append(const LatentGeom &g, const LatentDev &dv, const __half *C, const __half *Kr,
                                      const LatentTokens &a, cudaStream_t st);
// a: T and n[i] new tokens behind them (of Cn, Krn, [b][a.n_stride]); into [b][stride]
cudaError_t kivi_launch_latent_rows(const LatentGeom &g, const LatentDev &dv, const __half *Cn, const __half *Krn,
                                    __half *C, __half *Kr, const LatentTokens &a, int stride, int maxS, cudaStream_t st);
// The absorbed attention (kivi_latent_attn.cu); a: hq = hg = h, T, Tqk = Tqv =
// the quantized tokens, n, n_stride, and the work list of kivi_plan_latent.
constexpr int kLatRows = 64;   // rows of a row tile
constexpr int kLatFew = 32;    // ... where there are few
bool kivi_plan_latent(const LatentGeom &g, int h, ChunkArgs &a, int num_sms, ChunkPlan *plan);
size_t kivi_latent_partial_floats(const LatentGeom &g, int num_sms);
cudaError_t kivi_launch_latent_attn(const LatentGeom &g, const LatentDev &dv, const __half *Q, const __half *Qr,
                                    const __half *C, const __half *Kr, __half *O, ChunkArgs &a, const ChunkPlan &plan,
                                    float scale, float *partials, int device, int num_sms, cudaStream_t st);
// What the calls without a handle need of the current device: its number, SMs, and
// their status word (kivi_latent.cu; asked for once a device).  False: not available.
struct KiviDeviceInfo {
    int device, sms;
    unsigned *status;
};
bool kivi_device_info(KiviDeviceInfo *info);
// kivi_head_product, and kivi_latent_expanded_attn (T null: prompts), whose waits that
// run out show in *status (device; null: the device's word for calls without a handle)
kivi_status kivi_head_product_to(unsigned *status, const void *x, const void *w, int b, int h_x, int h, int n_stride,
                                 const int32_t *n, int K, int N, int transposed, void *out, kivi_stream_t stream);
kivi_status kivi_latent_expanded_to(unsigned *status, const void *q, const void *q_rope, const void *K, const void *Kr,
                                    const void *V, int b, int h, const int32_t *T, const int32_t *n, int n_stride,
                                    int s_stride, float scale, void *out, kivi_stream_t stream);
// Shared memory that a kernel may take, set once a device (done: a bit each).
template <typename K>
cudaError_t kivi_allow_smem(K *kernel, size_t bytes, int device, std::atomic<uint64_t> &done) {
    const uint64_t bit = 1ull << (device & 63);
    if (device < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && device < 64) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A launch as a programmatic dependent of the kernel before it on the stream: its
// CTAs are placed and set up while that one's last writes land, and wait
// (kivi_after_previous, every CTA, before any access to global memory and before it
// may return) until it is done.  Such a kernel reads by ordinary loads: those of the
// read-only path (const __restrict__ parameters, __ldg) ask for memory that nobody
// writes while the kernel runs, and the one before it still does.  The four kernels of
// a step for 64 sequences take 50 us for 51, the expanded form of short prompts 41 for
// 44, 1024 tokens over 8000 123 for 128.  cluster: CTAs of one.
template <typename... P, typename... A>
cudaError_t kivi_launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, int cluster,
                              A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}
#ifdef __CUDACC__
// EARLY: the kernel after this one may be placed as soon as all of this one's CTAs
// run, not only as they end (1024 tokens of 16 heads over 8000: 125.6 -> 123.1 us).
// So a kernel comes here with its tensor memory in hand: the next one's CTAs may take
// what is left, and wait for this kernel's end with it.
// Not after the attention over the cache and its join, whose successors would take
// places that they need (8 drafts of 5 over 16k: 45.3 us for 42.6).
template <bool EARLY = true>
__device__ __forceinline__ void kivi_after_previous() {
    if (EARLY) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif
