// kivi_head_product.cu -- a matrix of each head times rows of that head (or of
// all heads alike), on the 5th-generation tensor cores, and the entry point
// kivi_head_product: what latent attention does before and after itself.
//
// Mathematics.  out[i][e][s][:] = W_e x[i][e or 0][s][:] for head e and the
// tokens s < n[i] of sequence i, W_e [N][K] or, transposed, given as [K][N].
//   absorbing a query   qn [128] -> Wk_e^T qn [r]     K = 128, N = r, transposed
//   expanding a latent  c [r] -> Wk_e c, Wv_e c       K = r, N = 128, x of all heads
//   a head's output     ol [r] -> Wv_e ol             K = r, N = 128
//
// The rows of all sequences are one list (prefix sums of n), cut into tiles of
// 128, so that a step of 64 sequences of one token fills half a tile a head. A
// CTA makes 128 rows x 128 columns of one head: x W^T in tensor memory, 64 of K a
// stage; x by 16-byte asynchronous copies (any row of any sequence), W by TMA as
// the operand lies in memory, K-major or N-major, both in the 128-byte swizzle.
// Two CTAs an SM, so that one's first loads and last stores run under the other's
// products; with fewer CTAs than SMs one an SM and twice the stages, so that most
// of W is on its way at once.
//
// Rows that all heads share (a prompt's expansion) stay in shared memory, 128 of
// them up to 512 deep, while a CTA goes through several heads: W alone streams, the
// accumulator has two buffers, and one head's output is written under the next
// one's products.  (4096 tokens, 512 deep, 32 heads: 21.3 us, 0.81 PFLOP/s, where a
// CTA a tile, with twice the traffic from L2 and its own prologue, took 27.  A CTA
// takes in 128 KB of W for 128 columns; sent to two row tiles at once by multicast it
// took 24.4.)
#include "../../include/kivi.h"
#include "kivi_async.cuh"
#include "kivi_latent.cuh"
#include "kivi_mma.cuh"
#include "kivi_tcgen05.cuh"
#include "kivi_tma.cuh"

namespace {

constexpr int kHpRows = 128, kHpCols = 128, kHpK = 64;
constexpr int kHpThreads = 32 * 6;
constexpr unsigned kHpFull = 0xffffffffu;
constexpr int kHpA = kHpK * kHpRows * 2, kHpB = kHpK * kHpCols * 2;
__host__ __device__ constexpr size_t hp_smem(int stages) { return (size_t)stages * (kHpA + kHpB) + 1024; }

struct HeadArgs {
    const __half *x;
    __half *out;
    int b, hx, h, n_stride, K, N;
    int first[KIVI_MAX_BATCH + 1];   // rows before sequence i
    unsigned *status;
};

__device__ __forceinline__ void hp_copy16(void *dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
// sequence and token of row `row` of the list
__device__ __forceinline__ int2 hp_row(const HeadArgs &a, int row) {
    int lo = 0, hi = a.b;   // first[lo] <= row < first[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (a.first[m] <= row) lo = m;
        else hi = m;
    }
    return make_int2(lo, row - a.first[lo]);
}

// A row's 128 columns of the output (dst; null: no row) from the accumulator, a lane
// a row; read: called once they are read.  (Through shared memory, 64 consecutive
// bytes of 8 rows a store: no faster with many rows, 0.7 us slower with few.)
template <typename F>
__device__ __forceinline__ void hp_store(__half *dst, uint32_t acc, F read) {
#pragma unroll 1
    for (int c0 = 0; c0 < kHpCols; c0 += 32) {
        uint32_t o[32];
        tc_ld32(acc + c0, o);
        tc_wait_ld();
        if (c0 + 32 == kHpCols) read();
        if (dst)
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = h2u(__floats2half2_rn(__uint_as_float(o[c + 2 * k]), __uint_as_float(o[c + 2 * k + 1])));
                *reinterpret_cast<uint4 *>(dst + c0 + c) = make_uint4(v[0], v[1], v[2], v[3]);
            }
    }
}

// Warps 0-3: x's tiles, then the output; 4: W's tiles; 5: the products.
template <bool MN, int S>   // S: stages
__global__ void __launch_bounds__(kHpThreads, S > 3 ? 1 : 2)
    head_product_kernel(const __grid_constant__ HeadArgs a, const __grid_constant__ CUtensorMap tm) {
    extern __shared__ unsigned char raw[];
    unsigned char *sA = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u), *sB = sA + S * kHpA;
    __shared__ __align__(8) uint64_t bars[3 * S + 1];
    uint64_t *const bA = bars, *const bB = bA + S, *const eS = bB + S, *const bD = eS + S;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row0 = blockIdx.x * kHpRows, col0 = blockIdx.y * kHpCols, e = blockIdx.z;
    const int rows = a.first[a.b], nk = a.K / kHpK;
    if (tid < 3 * S + 1) {
        mbar_init(&bars[tid], tid < S ? 4 : 1);
        fence_mbar_init();
    }
    if (tid == 0) s_abort = 0;
    if (warp == 0) tc_alloc(&s_taddr, kHpCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    kivi_after_previous();
    const uint32_t taddr = s_taddr;
    const volatile int *abort = &s_abort;
    bool ok = true;

    if (warp < 4) {
        // x: a thread's 16-byte chunk of every 16th row
        constexpr int NR = kHpRows / 16;
        const __half *src[NR];
        unsigned in = 0;
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const int row = row0 + (tid >> 3) + 16 * k;
            if (row < rows) in |= 1u << k;
            const int2 p = hp_row(a, row < rows ? row : row0);
            src[k] = a.x + (((size_t)p.x * a.hx + (a.hx > 1 ? e : 0)) * a.n_stride + p.y) * a.K + 8 * (tid & 7);
        }
        const unsigned at = (tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) * 16);   // (16 rows further: the same chunk)
        auto told = [&](int it) {   // the stage's copies of this warp are in
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bA[it % S]);
        };
        for (int it = 0; it < nk && ok; ++it) {
            const int s = it % S;
            ok = __all_sync(kHpFull, it < S || mbar_wait_ab(&eS[s], (unsigned)(it / S + 1) & 1u, abort));
            if (!ok) break;
            unsigned char *dst = sA + s * kHpA + at;
#pragma unroll
            for (int k = 0; k < NR; ++k) hp_copy16(dst + k * 16 * 128, src[k] + it * kHpK, (in >> k) & 1u);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (it >= S - 2) {
                asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
                told(it - (S - 2));
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        for (int it = max(0, nk - (S - 2)); it < nk && ok; ++it) told(it);
        const int row = row0 + tid;
        const int2 p = hp_row(a, row < rows ? row : row0);
        ok = ok && __all_sync(kHpFull, mbar_wait_ab(bD, 0u, abort));
        if (ok) {
            tc_fence_after();
            hp_store(row < rows ? a.out + (((size_t)p.x * a.h + e) * a.n_stride + p.y) * a.N + col0 : nullptr,
                     taddr + ((uint32_t)(32 * warp) << 16), [] {});
            tc_fence_before();
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(a.status, KIVI_FLAG_WAIT);
        }
        __syncwarp();
    } else if (warp == 4) {
        if (lane == 0) {
            int it = 0;
            for (; it < nk; ++it) {
                const int s = it % S;
                ok = it < S || mbar_wait_ab(&eS[s], (unsigned)(it / S + 1) & 1u, abort);
                if (!ok) break;
                mbar_expect_tx(&bB[s], kHpB);
                unsigned char *dst = sB + s * kHpB;
                if (MN) {   // 64 of K x 64 columns, twice
                    tma_sw(dst, &tm, col0, e * a.K + it * kHpK, &bB[s]);
                    tma_sw(dst + kHpB / 2, &tm, col0 + 64, e * a.K + it * kHpK, &bB[s]);
                } else {
                    tma_sw(dst, &tm, it * kHpK, e * a.N + col0, &bB[s]);
                }
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(a.status, KIVI_FLAG_WAIT);
            }
            // every copy has landed before shared memory is given up (bounded)
            for (int y = max(0, it - S); y < it; ++y) mbar_wait(&bB[y % S], (unsigned)(y / S) & 1u);
        }
        __syncwarp();
    } else {
        constexpr uint32_t ID = tc_idesc_f16(kHpRows, kHpCols, MN ? 1 : 0);
        const uint64_t da = tc_desc_sw(sA, 16, 1024), db = MN ? tc_desc_sw(sB, kHpB / 2, 1024) : tc_desc_sw(sB, 16, 1024);
        int it = 0;
        for (; it < nk; ++it) {
            const int s = it % S;
            const unsigned ph = (unsigned)(it / S) & 1u;
            ok = __all_sync(kHpFull, mbar_wait_ab(&bA[s], ph, abort) && mbar_wait_ab(&bB[s], ph, abort));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kHpK / 16; ++c)
                tc_mma_f16_w(taddr, da + (uint32_t)((s * kHpA + 32 * c) >> 4),
                             db + (uint32_t)((s * kHpB + (MN ? 2048 : 32) * c) >> 4), ID, it > 0 || c > 0);
            tc_commit_w(&eS[s]);
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(a.status, KIVI_FLAG_WAIT);
        }
        // every product and commit is done before memory is given up (bounded)
        tc_commit_w(bD);
        for (int y = max(0, it - S); y < it; ++y) mbar_wait(&eS[y % S], (unsigned)(y / S) & 1u);
        mbar_wait(bD, 0u);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(taddr, kHpCols);
}

constexpr int kHsMaxK = 512;
__host__ __device__ constexpr int hs_stages(int C) { return C == 2 ? 3 : 5; }
__host__ __device__ constexpr size_t hs_smem(int C, int K) {
    return (size_t)kHpRows * K * 2 + (size_t)hs_stages(C) * C * kHpB + 1024;
}

// The rows of all heads alike: CTA (row tile, group) makes tiles [per y, per (y +
// 1)) of all heads' columns, 128 C a tile.  (Of 128 columns an MMA reads 8 KB of
// operands, 64 cycles of shared memory's bandwidth, for 64 cycles of work; of 256 12
// KB, 96 cycles, for 128.)  Warps as above.
template <int C>
__global__ void __launch_bounds__(kHpThreads, 1)
    head_product_shared_kernel(const __grid_constant__ HeadArgs a, const __grid_constant__ CUtensorMap tm, int per) {
    extern __shared__ unsigned char raw[];
    constexpr int S = hs_stages(C), NX = kHsMaxK / kHpK, Cols = C * kHpCols, B = C * kHpB;
    const int nk = a.K / kHpK, nc = a.N / kHpCols, cols = a.h * nc;
    unsigned char *sA = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u), *sB = sA + nk * kHpA;
    // counts 4: x in [64 of K], buffer read [buffer]; 1: the others
    constexpr int N4 = NX + 2, NB = N4 + 2 * S + 3;
    __shared__ __align__(8) uint64_t bars[NB];
    uint64_t *const bA = bars, *const eD = bars + NX, *const bB = bars + N4, *const eS = bB + S, *const bD = eS + S, *const bE = bD + 2;
    __shared__ uint32_t s_taddr;
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row0 = blockIdx.x * kHpRows, rows = a.first[a.b];
    const int j0 = blockIdx.y * per, j1 = min(j0 + per, (cols + C - 1) / C);
    if (tid < NB) {
        mbar_init(&bars[tid], tid < N4 ? 4 : 1);
        fence_mbar_init();
    }
    if (tid == 0) s_abort = 0;
    if (warp == 0) tc_alloc(&s_taddr, 2 * Cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    kivi_after_previous();
    const uint32_t taddr = s_taddr;
    const volatile int *abort = &s_abort;
    bool ok = true;

    if (warp < 4) {
        constexpr int NR = kHpRows / 16;
        const unsigned at = (tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) * 16);
        const __half *src[NR];
        unsigned in = 0;
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            const int row = row0 + (tid >> 3) + 16 * k;
            if (row < rows) in |= 1u << k;
            const int2 p = hp_row(a, row < rows ? row : row0);
            src[k] = a.x + ((size_t)p.x * a.n_stride + p.y) * a.K + 8 * (tid & 7);
        }
        for (int it = 0; it < NX; ++it) {   // (past K: empty groups)
#pragma unroll
            for (int k = 0; k < NR; ++k)
                if (it < nk) hp_copy16(sA + it * kHpA + at + k * 16 * 128, src[k] + it * kHpK, (in >> k) & 1u);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        auto told = [&](int it) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && it < nk) mbar_arrive(&bA[it]);
        };
        static_assert(NX == 8, "a wait for each group");
        asm volatile("cp.async.wait_group 7;" ::: "memory"); told(0);
        asm volatile("cp.async.wait_group 6;" ::: "memory"); told(1);
        asm volatile("cp.async.wait_group 5;" ::: "memory"); told(2);
        asm volatile("cp.async.wait_group 4;" ::: "memory"); told(3);
        asm volatile("cp.async.wait_group 3;" ::: "memory"); told(4);
        asm volatile("cp.async.wait_group 2;" ::: "memory"); told(5);
        asm volatile("cp.async.wait_group 1;" ::: "memory"); told(6);
        asm volatile("cp.async.wait_group 0;" ::: "memory"); told(7);
        const int row = row0 + tid;
        const int2 p = hp_row(a, row < rows ? row : row0);
        for (int j = j0; j < j1 && ok; ++j) {
            const int y = j - j0, b = y & 1;
            ok = __all_sync(kHpFull, mbar_wait_ab(&bD[b], (unsigned)(y >> 1) & 1u, abort));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < C; ++k) {
                const int e = (C * j + k) / nc, col0 = (C * j + k - e * nc) * kHpCols;
                hp_store(row < rows && C * j + k < cols ? a.out + (((size_t)p.x * a.h + e) * a.n_stride + p.y) * a.N + col0 : nullptr,
                         taddr + ((uint32_t)(32 * warp) << 16) + Cols * b + kHpCols * k, [&] {   // the buffer is read
                             if (k < C - 1) return;
                             tc_fence_before();
                             __syncwarp();
                             if (lane == 0) mbar_arrive(&eD[b]);
                         });
            }
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(a.status, KIVI_FLAG_WAIT);
        }
        __syncwarp();
    } else if (warp == 4) {
        if (lane == 0) {
            int it = 0;
            const int end = (j1 - j0) * nk;
            for (; it < end; ++it) {
                const int s = it % S, j = j0 + it / nk;
                ok = it < S || mbar_wait_ab(&eS[s], (unsigned)(it / S + 1) & 1u, abort);
                if (!ok) break;
                mbar_expect_tx(&bB[s], B);
                tma_sw(sB + s * B, &tm, it % nk * kHpK, j * Cols, &bB[s]);
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(a.status, KIVI_FLAG_WAIT);
            }
            // every copy has landed before shared memory is given up (bounded)
            for (int y = max(0, it - S); y < it; ++y) mbar_wait(&bB[y % S], (unsigned)(y / S) & 1u);
        }
        __syncwarp();
    } else {
        constexpr uint32_t ID = tc_idesc_f16(kHpRows, Cols, 0);
        const uint64_t da = tc_desc_sw(sA, 16, 1024), db = tc_desc_sw(sB, 16, 1024);
        int s = 0, it = 0;
        unsigned ph = 0;
        for (int j = j0; j < j1 && ok; ++j) {
            const int y = j - j0, b = y & 1;
            // the buffer's last output is read
            ok = __all_sync(kHpFull, y < 2 || mbar_wait_ab(&eD[b], (unsigned)((y >> 1) + 1) & 1u, abort));
            for (int k = 0; k < nk && ok; ++k, ++it) {
                ok = __all_sync(kHpFull, (y > 0 || mbar_wait_ab(&bA[k], 0u, abort)) && mbar_wait_ab(&bB[s], ph, abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kHpK / 16; ++c)
                    tc_mma_f16_w(taddr + Cols * b, da + (uint32_t)((k * kHpA + 32 * c) >> 4),
                                 db + (uint32_t)((s * B + 32 * c) >> 4), ID, k > 0 || c > 0);
                tc_commit_w(&eS[s]);
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (ok) tc_commit_w(&bD[b]);
        }
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(a.status, KIVI_FLAG_WAIT);
        }
        // every product and commit is done before memory is given up (bounded)
        tc_commit_w(bE);
        mbar_wait(bE, 0u);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(taddr, 2 * Cols);
}

kivi_status fail(kivi_status s, const char *msg) {
    kivi_set_last_error(msg);
    return s;
}

}  // namespace

kivi_status kivi_head_product_to(unsigned *status, const void *x, const void *w, int b, int h_x, int h, int n_stride,
                                 const int32_t *n, int K, int N, int transposed, void *out, kivi_stream_t stream) {
    if (b < 1 || h < 1 || n_stride < 0 || K < 1 || N < 1) return fail(KIVI_ERR_INVALID_ARG, "sizes must be positive");
    if (h_x != 1 && h_x != h) return fail(KIVI_ERR_INVALID_ARG, "h_x must be 1 or h");
    if (b > KIVI_MAX_BATCH) return fail(KIVI_ERR_UNSUPPORTED, "b above 1024");
    if (h > 1024) return fail(KIVI_ERR_UNSUPPORTED, "more than 1024 heads");
    if (K % kHpK != 0 || N % kHpCols != 0 || K > 16384 || N > 16384)
        return fail(KIVI_ERR_UNSUPPORTED, "K must be a multiple of 64 and N of 128, at most 16384");
    if (!n) return fail(KIVI_ERR_INVALID_ARG, "n is null");
    HeadArgs a;
    long long rows = 0;
    for (int i = 0; i < b; ++i) {
        if (n[i] < 0 || n[i] > n_stride) return fail(KIVI_ERR_INVALID_ARG, "n[i] outside [0, n_stride]");
        a.first[i] = (int)rows;
        rows += n[i];
        if (rows > (1LL << 30)) return fail(KIVI_ERR_UNSUPPORTED, "more than 2^30 tokens");
    }
    a.first[b] = (int)rows;
    if (rows == 0) return KIVI_OK;
    if (!x || !w || !out) return fail(KIVI_ERR_INVALID_ARG, "a tensor pointer is null");
    if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)out) & 15u)
        return fail(KIVI_ERR_INVALID_ARG, "x, w and out must be 16-byte aligned");
    a.x = (const __half *)x;
    a.out = (__half *)out;
    a.b = b;
    a.hx = h_x;
    a.h = h;
    a.n_stride = n_stride;
    a.K = K;
    a.N = N;
    KiviDeviceInfo info;
    if (!kivi_device_info(&info)) return fail(KIVI_ERR_CUDA, "no status word on the current device");
    a.status = status ? status : info.status;
    const bool mn = transposed != 0;
    const dim3 grid((unsigned)((rows + kHpRows - 1) / kHpRows), (unsigned)(N / kHpCols), (unsigned)h);
    const int cols = h * (N / kHpCols);   // column tiles of all heads
    const bool shared = h_x == 1 && h > 1 && !mn && K <= kHsMaxK && (long long)grid.x * cols > info.sms;
    // (shared) a CTA an SM: as many groups of heads as leave every row tile one, and
    // the tiles of C column tiles that each then has.  C = 2 where that leaves no CTA
    // more columns, and several tiles (4096 tokens, 32 heads: 21.3 us for 22.7; 3000, 11
    // heads, 256 deep, in tiles of one 8.8 for 9.8)
    const auto share = [&](int C) {
        const long long tiles = (cols + C - 1) / C;
        long long groups = info.sms / (long long)grid.x;
        if (groups < 1) groups = 1;
        if (groups > tiles) groups = tiles;
        return (int)((tiles + groups - 1) / groups);
    };
    const int C = share(1) >= 4 && 2 * share(2) <= share(1) ? 2 : 1;
    CUtensorMap tm;
    cudaError_t e = mn ? make_sw_map(&tm, (const __half *)w, (long long)h * K, N, kHpK)
                       : make_sw_map(&tm, (const __half *)w, (long long)h * N, K, shared ? C * kHpCols : kHpCols);
    if (e == cudaSuccess && shared) {
        const int tiles = (cols + C - 1) / C, per = share(C);
        static std::atomic<uint64_t> done[2];
        const auto kernel = C == 2 ? head_product_shared_kernel<2> : head_product_shared_kernel<1>;
        e = kivi_allow_smem(kernel, hs_smem(C, kHsMaxK), info.device, done[C - 1]);
        if (e == cudaSuccess)
            e = kivi_launch_after(kernel, dim3(grid.x, (unsigned)((tiles + per - 1) / per)), kHpThreads, hs_smem(C, K),
                                  (cudaStream_t)stream, 1, a, tm, per);
        return e == cudaSuccess ? KIVI_OK : fail(KIVI_ERR_CUDA, cudaGetErrorString(e));
    }
    const bool deep = K > 2 * kHpK && (long long)grid.x * grid.y * grid.z <= info.sms;
    const auto kernel = deep ? (mn ? head_product_kernel<true, 6> : head_product_kernel<false, 6>)
                             : (mn ? head_product_kernel<true, 3> : head_product_kernel<false, 3>);
    const size_t smem = hp_smem(deep ? 6 : 3);
    static std::atomic<uint64_t> done[4];
    if (e == cudaSuccess) e = kivi_allow_smem(kernel, smem, info.device, done[2 * deep + mn]);
    if (e != cudaSuccess) return fail(KIVI_ERR_CUDA, cudaGetErrorString(e));
    e = kivi_launch_after(kernel, grid, kHpThreads, smem, (cudaStream_t)stream, 1, a, tm);
    return e == cudaSuccess ? KIVI_OK : fail(KIVI_ERR_CUDA, cudaGetErrorString(e));
}

extern "C" kivi_status kivi_head_product(const void *x, const void *w, int b, int h_x, int h, int n_stride,
                                         const int32_t *n, int K, int N, int transposed, void *out,
                                         kivi_stream_t stream) {
    kivi_set_last_error("");
    return kivi_head_product_to(nullptr, x, w, b, h_x, h, n_stride, n, K, N, transposed, out, stream);
}
