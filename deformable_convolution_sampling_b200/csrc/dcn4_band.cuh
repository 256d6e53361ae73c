// dcn4_band.cuh — what the kernels of the attention-layer operators share: the
// geometry of the band attention (which keys a query sees, the tiles of keys a
// block of queries has to visit) and the launchers the C ABI calls.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dcn4 {

// Distances and positions stay far from the ends of 32-bit integers: sequences
// are shorter than kBandMaxLen, the first query's position is clamped to
// +-kBandMaxLen, and "unlimited" is a window no pair exceeds.
constexpr int kBandMaxLen = 1 << 28;
constexpr int kBandFar = 1 << 30;
constexpr int kBandMaxReach = 1024;    // relative positions with buckets of their own: -M..M, M at most this
constexpr int kBandMaxBuckets = 1024;
constexpr int kBandSms = 148;          // B200: SMs a launch should fill (sizes workspaces too, so a constant)

// One call of the band attention.  Query i of image n stands at position
// start(n) + i; key j is seen by position p iff j < klen(n), j - p <= right and
// (p - j <= left or j < sinks).
struct BandArgs {
    int N, Lq, Lk, Hq, Hk, G, D;  // G = Hq / Hk query heads share a key head
    int left, right, sinks;       // kBandFar: no limit
    float scale;
    int nb, M;                    // relative bias: nb buckets (0: none), reach M
    int dtype;
    long long q_batch, q_row, k_batch, k_row, v_batch, v_row;  // elements between images and tokens
    const void *q, *k, *v;
    const void* bias;             // [nb, Hq]
    const int* buckets;           // [2 M + 1], of relative position -M..M
    const int *q_start, *q_len, *k_len;  // [N] or NULL
};

__device__ __forceinline__ int band_klen(const BandArgs& a, int n) {
    return a.k_len ? max(0, min(a.k_len[n], a.Lk)) : a.Lk;
}
__device__ __forceinline__ int band_qlen(const BandArgs& a, int n) {
    return a.q_len ? max(0, min(a.q_len[n], a.Lq)) : a.Lq;
}
__device__ __forceinline__ int band_start(const BandArgs& a, int n) {
    return a.q_start ? max(-kBandMaxLen, min(a.q_start[n], kBandMaxLen)) : a.Lk - a.Lq;
}
__device__ __forceinline__ bool band_sees(const BandArgs& a, int p, int j, int klen) {
    return j < klen && j - p <= a.right && (p - j <= a.left || j < a.sinks);
}

// What the backward subtracts from a row's scores.  A row whose log sum is -infinity
// has probabilities of 0, also where a bias of -infinity makes s - lse a NaN.
__device__ __forceinline__ float band_lse_ref(float lse) { return lse == -INFINITY ? INFINITY : lse; }
// One number in 32 bits holds a row's log sum to 2^-24 of itself.  Where that is far from
// zero (a row that sees only keys of the type's lowest bias keeps nothing of its log l),
// e^(s - lse) is off by a factor, and the backward takes the row's maximum m and sum l
// anew: p = e^(s - m) / l.  Up to 512 the factor is within 2^-15 of 1, a sixteenth of
// fp16's half step and no more than the rounding of such a score itself.
constexpr float kBandFarLse = 512.f;
__device__ __forceinline__ bool band_far(float ref) { return fabsf(ref) > kBandFarLse && fabsf(ref) < INFINITY; }

// The tiles of `bn` keys that positions p_lo..p_hi (all of them queries) have to
// visit: the tiles of the sinks, then those of the window.
struct BandTiles {
    int sink, lo, hi;  // tiles [0, sink) and [lo, hi)
    __device__ __forceinline__ int count() const { return sink + hi - lo; }
    __device__ __forceinline__ int tile(int t) const { return t < sink ? t : lo + t - sink; }
};
__device__ __forceinline__ BandTiles band_tiles(const BandArgs& a, int p_lo, int p_hi, int klen, int bn) {
    const int hi = min(klen, p_hi + a.right + 1);  // p_hi < 2^29, right <= 2^30: no overflow
    const int lo = max(0, p_lo - a.left);
    const int sink = max(0, min(a.sinks, hi));
    BandTiles t;
    t.sink = (sink + bn - 1) / bn;
    if (lo < hi) {
        t.lo = lo / bn;
        t.hi = (hi + bn - 1) / bn;
        t.sink = min(t.sink, t.lo);
    } else {
        t.lo = t.hi = t.sink;
    }
    return t;
}
// The queries [lo, hi) of image n that see some key of [k0, k1).
__device__ __forceinline__ void band_queries(const BandArgs& a, int start, int qlen, int k0, int k1, int& lo, int& hi) {
    lo = max(0, k0 - a.right - start);
    hi = k0 < a.sinks ? qlen : min(qlen, k1 + a.left - start);  // k1 + left < 2^31
    if (lo > hi) lo = hi;
}

// Bytes of scratch (see the C ABI), each a multiple of 256.
size_t band_forward_workspace_bytes(const BandArgs& a);
size_t band_backward_workspace_bytes(const BandArgs& a, bool want_bias);
// The status words of the kernels with bounded waits, or-ed.
cudaError_t band_status(unsigned* status, bool reset);
// out = 0 and lse = -infinity (no keys at all).
cudaError_t launch_band_empty(const BandArgs& a, void* out, float* lse, cudaStream_t stream);
cudaError_t launch_band_forward(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream);
cudaError_t launch_band_backward(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq,
                                 void* gk, void* gv, void* gbias, void* ws, cudaStream_t stream);

// RMS norm of query and key heads and the position rotation (dcn4_qknorm.cu).
struct QkNormArgs {
    int N, L, Hq, Hk, D, R, axes, interleaved, dtype;
    float eps;
    long long q_batch, q_row, k_batch, k_row;
    const void *q, *k, *wq, *wk;
    const float *pos, *inv_freq;
};
size_t qknorm_backward_workspace_bytes(const QkNormArgs& a);
cudaError_t launch_qknorm_forward(const QkNormArgs& a, void* qo, void* ko, cudaStream_t stream);
cudaError_t launch_qknorm_backward(const QkNormArgs& a, const void* gqo, const void* gko, void* gq, void* gk,
                                   void* gwq, void* gwk, void* ws, cudaStream_t stream);

}  // namespace dcn4
