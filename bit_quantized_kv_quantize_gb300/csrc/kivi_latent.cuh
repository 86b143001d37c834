// kivi_latent.cuh -- what the host and the kernels of the latent cache share:
// its geometry and layout, and the launchers.
//
// Per sequence the cache holds each token's latent vector c [r] and rotary key
// kr [64].  Tokens [0, Tq) are quantized, a token's groups of G channels with an
// fp16 scale and zero each (the value side of the KIVI quantizer); the newest
// R, [Tq, T), are fp16.  Device memory, tokens in blocks of 64 (R and the
// capacity are multiples of 64, so a block of tokens is a block of memory):
//   records  [b][blocks]: codes, then scales and zeros.  16-byte words of codes
//            [r bits / 128][64 tokens]: word x of a token covers channels
//            (128 / bits) x ..  In each 32-bit word (16-bit half h, field f of
//            `bits` bits) is the code of channel 2 f + h of the word's 32 /
//            bits.  Scale and zero, a half2, [r / G][64 tokens].
//   ring     [b][R / 64] and rotary keys [b][blocks]: fp16 blocks in the tensor
//            cores' core-matrix layout, [channels / 8][64 tokens][8 channels]:
//            a block is copied into an attention tile as it is.  Token tau of
//            the ring is at block (tau / 64) mod (R / 64).
#pragma once
#include "kivi_chunk.cuh"
#include "kivi_internal.cuh"

constexpr int kLatRope = 64;    // channels of the rotary key
constexpr int kLatHead = 128;   // channels of a head's other keys, and of its values

struct LatentGeom {
    int b, r, bits, G, R;
    int blocks;      // of 64 tokens, a sequence
    int off_sz;      // scales and zeros in a record (bytes)
    int rec_bytes;
};
struct LatentDev {
    unsigned char *rec;
    __half *ring, *kr;
    unsigned *status;
};

__host__ __device__ __forceinline__ size_t lat_rec(const LatentGeom &g, int i, int kb) {
    return ((size_t)i * g.blocks + kb) * g.rec_bytes;
}
// a block of the ring, of the rotary keys (halves)
__host__ __device__ __forceinline__ size_t lat_ring(const LatentGeom &g, int i, int kb) {
    const int nr = g.R / KIVI_KBLK;
    return ((size_t)i * nr + kb % nr) * KIVI_KBLK * g.r;
}
__host__ __device__ __forceinline__ size_t lat_kr(const LatentGeom &g, int i, int kb) {
    return ((size_t)i * g.blocks + kb) * KIVI_KBLK * kLatRope;
}
// quantized tokens of T
__host__ __device__ __forceinline__ int lat_tq(int T, int R) { return T > R ? T - R : 0; }

// n[i] tokens at positions T[i].. (counts from the host mirror)
struct LatentTokens {
    int n_stride;
    int T[KIVI_MAX_BATCH], n[KIVI_MAX_BATCH];
};

cudaError_t kivi_launch_latent_append(const LatentGeom &g, const LatentDev &dv, const __half *C, const __half *Kr,
                                      const LatentTokens &a, int maxn, cudaStream_t st);
cudaError_t kivi_launch_latent_restore(const LatentGeom &g, const LatentDev &dv, __half *C, __half *Kr,
                                       const LatentTokens &a, int maxT, cudaStream_t st);
// The absorbed attention (kivi_latent_attn.cu); a: hq = hg = h, T, Tqk = Tqv =
// the quantized tokens, n, n_stride, and the work list of kivi_plan_latent.
constexpr int kLatRows = 64;   // rows of a row tile
bool kivi_plan_latent(const LatentGeom &g, int h, ChunkArgs &a, int num_sms, ChunkPlan *plan);
size_t kivi_latent_partial_floats(const LatentGeom &g, int num_sms);
cudaError_t kivi_launch_latent_attn(const LatentGeom &g, const LatentDev &dv, const __half *Q, const __half *Qr,
                                    const __half *C, const __half *Kr, __half *O, ChunkArgs &a, const ChunkPlan &plan,
                                    float scale, float *partials, int num_sms, cudaStream_t st);
// The status word of the calls without a handle, on the current device
// (kivi_latent.cu); null: not available.
unsigned *kivi_device_status();
