// kivi_latent_places.h -- which warp of an append to the latent cache reads and
// writes which places of a sequence's ring.  Whole numbers only: the kernel and a
// host compiler take the same lines.
#pragma once

#ifdef __CUDACC__
#define KIVI_PLACES __host__ __device__ __forceinline__
#else
#define KIVI_PLACES inline
#endif

constexpr int kLatTok = 128;    // tokens of a block

// quantized tokens of T
KIVI_PLACES int lat_tq(int T, int R) { return T > R ? T - R : 0; }

// Where an append of n > 0 tokens ends in the ring: behind them, or, where it begins
// their last block, with that block, whose places behind the last token are set to
// zero.  (Attention multiplies them with weights of zero, and what an earlier use of
// the cache left there need not be finite.)
KIVI_PLACES int lat_end(int T, int n) {
    const int last = (T + n - 1) / kLatTok * kLatTok;   // the last block's first token
    return last >= T ? last + kLatTok : T + n;
}

// What warp x does, 0 <= x < lat_end - T, that of token tau = T + x (a new one below T +
// n, else a place to set to zero); W places (a multiple of 128, R + 128 or more), token
// o's is o mod W.  The window of R moves from Tq to Tq1; B is the first token of Tq1's
// block, from which on the ring keeps every token (those before Tq1 as their codes
// restore them).
//
// So the places of [first, end), first = max(T, B), are written, of W tokens at most:
// each by its token's warp, which first quantizes the cached token there that leaves
// the window (`under`, several times W before; n may be larger than W).  The other
// cached tokens that leave, whose places are not written, are the warps' in turn
// (`own`, the x-th of warp x), and are written back there if they lie in [B, Tq1).  No
// warp reads or writes a place that another writes.  (tests/test_latent_places.py walks
// these lines.)
struct LatMoves {
    int own;     // cached token that it quantizes from the ring (-1: none)
    int under;   // another one, whose place its own token takes, before it does (-1: none)
    bool codes;  // its own token is quantized (else it goes into the ring as it is)
};
KIVI_PLACES LatMoves lat_moves(int T, int n, int R, int W, int x) {
    const int tau = T + x, Tq = lat_tq(T, R), Tq1 = lat_tq(T + n, R), B = Tq1 / kLatTok * kLatTok;
    const int first = T > B ? T : B, leaves = T < Tq1 ? T : Tq1;   // cached tokens [Tq, leaves) leave
    LatMoves m = {-1, -1, tau < Tq1};
    if (Tq < leaves) {
        const int own = Tq + x, under = tau - (x + W) / W * W;   // (the last token before T in tau's place)
        if (own < leaves && own + (first - own + W - 1) / W * W >= lat_end(T, n)) m.own = own;
        if (tau >= first && under >= Tq) m.under = under;
    }
    return m;
}
// whether token o, quantized by this append, is written into its place too
KIVI_PLACES bool lat_restored(int T, int n, int R, int o) { return o / kLatTok == lat_tq(T + n, R) / kLatTok; }
