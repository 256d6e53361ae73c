// dcn4_band_parts.cuh — the band attention's partial results (a long key axis
// split over CTAs, the bias gradient's part of every CTA), the kernels that join
// them, and the launchers of its forms.  Internal to the band attention.
#pragma once

#include <algorithm>

#include "dcn4_band.cuh"

namespace dcn4 {

// Partial forwards over ranges of the keys: of row r = (n Hq + h) Lq + i and
// range s, the unnormalised output o[r splits + s][D] with its running maximum
// and sum ml[r splits + s].
struct BandPart {
    float* o;
    float2* ml;
};
__host__ __device__ inline long long band_rows(const BandArgs& a) { return static_cast<long long>(a.N) * a.Hq * a.Lq; }
inline size_t band_part_bytes(const BandArgs& a, int splits) {
    return splits > 1 ? static_cast<size_t>(band_rows(a)) * splits * (a.D * sizeof(float) + sizeof(float2)) : 0;
}
inline BandPart band_part(const BandArgs& a, int splits, void* ws) {
    BandPart p;
    p.o = static_cast<float*>(ws);  // rows of D floats: 16-byte aligned
    p.ml = reinterpret_cast<float2*>(p.o + band_rows(a) * splits * a.D);
    return p;
}

// Ranges of the keys for `ctas` CTAs whose `queries` neighbouring queries visit
// tiles of `bn` keys: enough to put `per_sm` CTAs on every SM, none shorter than
// four tiles (the join reads a row of fp32 a range back).
inline int band_splits(const BandArgs& a, long long ctas, int queries, int bn, int per_sm) {
    const long long span = std::min<long long>(a.Lk, static_cast<long long>(std::min(a.left, kBandMaxLen)) +
                                                         std::min(a.right, kBandMaxLen) + queries + a.sinks);
    const long long tiles = (span + bn - 1) / bn;
    const long long want = (static_cast<long long>(per_sm) * kBandSms + ctas - 1) / std::max<long long>(ctas, 1);
    return static_cast<int>(std::max<long long>(1, std::min<long long>(std::min<long long>(want, tiles / 4), 256)));
}

// Where a row sees no more keys than this, what meets them (probabilities and their
// gradients) keeps more than the I/O type's bits on the tensor cores: few roundings do
// not average out, and a small call's time is not in its products.
constexpr int kBandExactKeys = 64;
// The most keys that a row can see.
inline long long band_most_keys(const BandArgs& a) {
    return std::min<long long>(a.Lk, static_cast<long long>(std::min(a.left, kBandMaxLen)) + std::min(a.right, kBandMaxLen) + 1 + a.sinks);
}

// out and lse of every row from its parts, whose maxima are in `unit` natural units (1, or ln 2 of base 2).
cudaError_t launch_band_join(const BandArgs& a, int splits, BandPart part, float unit, void* out, float* lse, cudaStream_t stream);
// gbias from sums of ds along diagonals: diag[((n Hk + hk) per + c) each + w][G][2 M + 1], c < per
// CTAs of an image and key head, w < each sums a CTA.  Needs band_sum_bytes of scratch.
size_t band_sum_bytes(const BandArgs& a);
cudaError_t launch_band_bias_sum(const BandArgs& a, int per, int each, const float* diag, float* sums, void* gbias,
                                 cudaStream_t stream);

// 16-bit types on the tensor cores (dcn4_band_fwd_tc.cu).
size_t band_fwd_tc_part_bytes(const BandArgs& a);
cudaError_t launch_band_fwd_tc(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream);
cudaError_t band_fwd_status(unsigned* status, bool reset);

// 16-bit types, up to 16 rows (dcn4_band_few.cu).
bool band_few_fits(const BandArgs& a);
size_t band_few_part_bytes(const BandArgs& a);
cudaError_t launch_band_few(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream);

// 16-bit backward on the tensor cores (dcn4_band_bwd_tc.cu).
size_t band_bwd_tc_workspace(const BandArgs& a, bool want_bias);
cudaError_t launch_band_bwd_tc(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq, void* gk, void* gv,
                               void* gbias, void* ws, cudaStream_t stream);
cudaError_t band_bwd_status(unsigned* status, bool reset);

// fp32, on the fp32 pipes (dcn4_band_simt.cu).
int simt_row_blocks(const BandArgs& a);
int simt_splits(const BandArgs& a);
cudaError_t launch_band_simt_forward(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream);
cudaError_t launch_band_simt_backward(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq,
                                      void* gk, void* gv, void* gbias, void* ws, cudaStream_t stream);
size_t band_simt_backward_workspace(const BandArgs& a, bool want_bias);

}  // namespace dcn4
