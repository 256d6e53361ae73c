// dcn4_band.cu — the band attention's dispatch, workspaces, and the kernels that
// join partial results.
#include <cmath>

#include "dcn4_band_parts.cuh"
#include "dcn4_common.cuh"

namespace dcn4 {
namespace {

// out = (sum_s o_s e^(m_s - m)) / (sum_s l_s e^(m_s - m)), lse = m + log of that
// sum: a warp per row.  The m_s come in the unit that their kernel holds scores in (`unit`
// natural ones): a conversion would round each on its own, and where scores are of 10^6 the
// parts' weights with it.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(BandArgs a, int splits, BandPart part, float unit, T* __restrict__ out,
                                                   float* __restrict__ lse, long long rows) {
    const long long r = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    // a lane per part for the factors, a lane per entry for the sums; sixteen parts' loads go out before
    // anything waits for them (one batch mostly: the kernel is a launch and two latencies)
    constexpr int U = 16;
    const float2* ml = part.ml + r * splits;
    const float* po = part.o + r * splits * a.D + lane;
    float x[U][4];
    auto fetch = [&](int s) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                x[u][c] = s + u < splits && lane + 32 * c < a.D ? __ldg(po + static_cast<long long>(s + u) * a.D + 32 * c) : 0.f;
    };
    fetch(0);
    float2 v = lane < splits ? __ldg(ml + lane) : make_float2(-INFINITY, 0.f);
    float m = v.x;
    for (int s = 32 + lane; s < splits; s += 32) m = fmaxf(m, __ldg(ml + s).x);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[4] = {};
    for (int s0 = 0; s0 < splits; s0 += 32) {
        if (s0) v = s0 + lane < splits ? __ldg(ml + s0 + lane) : make_float2(0.f, 0.f);
        const float mine = v.y != 0.f ? expf((v.x - ref) * unit) : 0.f;  // a range may hold nothing the row sees
        l += v.y * mine;
        for (int s = s0; s < min(s0 + 32, splits); s += U) {
            if (s) fetch(s);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float f = __shfl_sync(0xffffffffu, mine, (s + u - s0) & 31);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (f != 0.f && s + u < splits) o[c] = fmaf(x[u][c], f, o[c]);
            }
        }
    }
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    const int i = static_cast<int>(r % a.Lq);
    const long long nh = r / a.Lq, n = nh / a.Hq, h = nh - n * a.Hq;
    const float f = l == 0.f ? 0.f : 1.f / l;
    T* to = out + ((n * a.Lq + i) * a.Hq + h) * a.D;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (lane + 32 * c < a.D) to[lane + 32 * c] = from_f32<T>(o[c] * f);
    if (lane == 0) lse[r] = l == 0.f ? -INFINITY : m * unit + logf(l);
}

// sums[z][h][rel] = the diagonal sums of head h, in a fixed order; `chunk` CTAs' a block.
// 2^shift sums a CTA, `per` CTAs an image and key head, `all` of them for a key head.
__global__ void __launch_bounds__(256) diag_sum_kernel(BandArgs a, unsigned all, unsigned per, unsigned chunk, int shift,
                                                       const float* __restrict__ diag, float* __restrict__ sums) {
    __shared__ float s_part[8][32];
    constexpr int U = 8;  // loads at a time, also in the last batch
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.x, len = 2 * a.M + 1, rel = blockIdx.y * 32 + lane;
    const unsigned hk = h / a.G, g = h - hk * a.G, c0 = blockIdx.z * chunk, c1 = min(all, c0 + chunk);
    const long long row = static_cast<long long>(a.G) * len;
    const float* from = diag + static_cast<long long>(g) * len + rel;
    float s = 0.f;
    for (unsigned c = c0; c < c1; c += (8 * U) >> shift) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned x = warp + 8 * u, q = c + (x >> shift), n = q / per;
            const unsigned cta = (n * a.Hk + hk) * per + (q - n * per);  // a grid: 31 bits
            v[u] = q < c1 && rel < len ? __ldg(from + ((static_cast<long long>(cta) << shift) + (x & ((1u << shift) - 1u))) * row) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) s += v[u];
    }
    s_part[warp][lane] = s;
    __syncthreads();
    if (warp || rel >= len) return;
    for (int w = 1; w < 8; ++w) s += s_part[w][lane];
    sums[(static_cast<long long>(blockIdx.z) * a.Hq + h) * len + rel] = s;
}

// gbias[b][h], b of a block's 64: head h's sums by relative position into shared memory,
// then a warp sums those of its bucket.
template <typename T>
__global__ void __launch_bounds__(256) bucket_sum_kernel(BandArgs a, int parts, const float* __restrict__ sums, T* __restrict__ gbias) {
    __shared__ float s_sum[2 * kBandMaxReach + 1];
    const int h = blockIdx.x, len = 2 * a.M + 1, lane = threadIdx.x & 31;
    for (int r = threadIdx.x; r < len; r += 256) {
        float s = 0.f;
        for (int z0 = 0; z0 < parts; z0 += 16) {
            float v[16];
#pragma unroll
            for (int z = 0; z < 16; ++z) v[z] = z0 + z < parts ? __ldg(sums + (static_cast<long long>(z0 + z) * a.Hq + h) * len + r) : 0.f;
#pragma unroll
            for (int z = 0; z < 16; ++z) s += v[z];
        }
        s_sum[r] = s;
    }
    __syncthreads();
    for (int b = blockIdx.y * 64 + (threadIdx.x >> 5); b < min(a.nb, static_cast<int>(blockIdx.y + 1) * 64); b += 8) {
        float s = 0.f;
        for (int r = lane; r < len; r += 32)
            if (__ldg(a.buckets + r) == b) s += s_sum[r];
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) gbias[static_cast<long long>(b) * a.Hq + h] = from_f32<T>(s);
    }
}

__global__ void __launch_bounds__(256) no_keys_kernel(float* __restrict__ lse, long long rows) {
    const long long r = blockIdx.x * 256ll + threadIdx.x;
    if (r < rows) lse[r] = -INFINITY;
}

constexpr unsigned kSumParts = 32;  // blocks a diagonal's sum is shared by, at most

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_band_join(const BandArgs& a, int splits, BandPart part, float unit, void* out, float* lse, cudaStream_t stream) {
    const long long rows = band_rows(a);
    const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
    switch (a.dtype) {
        case 0: join_kernel<float><<<grid, 256, 0, stream>>>(a, splits, part, unit, static_cast<float*>(out), lse, rows); break;
        case 1: join_kernel<__half><<<grid, 256, 0, stream>>>(a, splits, part, unit, static_cast<__half*>(out), lse, rows); break;
        case 2: join_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, splits, part, unit, static_cast<__nv_bfloat16*>(out), lse, rows); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

size_t band_sum_bytes(const BandArgs& a) {
    return static_cast<size_t>(kSumParts) * a.Hq * (2 * a.M + 1) * sizeof(float);
}

cudaError_t launch_band_bias_sum(const BandArgs& a, int per, int each, const float* diag, float* sums, void* gbias,
                                 cudaStream_t stream) {
    const int shift = each == 1 ? 0 : 4;  // one sum a CTA, or sixteen
    const unsigned all = static_cast<unsigned>(a.N) * per, batch = 64u >> shift;
    const unsigned chunk = std::max((all + kSumParts * batch - 1) / (kSumParts * batch), 1u) * batch, zs = (all + chunk - 1) / chunk;
    // (heads along x: the other dimensions of a grid end at 65535)
    diag_sum_kernel<<<dim3(a.Hq, (2 * a.M + 32) / 32, zs), 256, 0, stream>>>(a, all, per, chunk, shift, diag, sums);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const dim3 grid(a.Hq, (a.nb + 63) / 64);
    switch (a.dtype) {
        case 0: bucket_sum_kernel<float><<<grid, 256, 0, stream>>>(a, static_cast<int>(zs), sums, static_cast<float*>(gbias)); break;
        case 1: bucket_sum_kernel<__half><<<grid, 256, 0, stream>>>(a, static_cast<int>(zs), sums, static_cast<__half*>(gbias)); break;
        case 2: bucket_sum_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, static_cast<int>(zs), sums, static_cast<__nv_bfloat16*>(gbias)); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

cudaError_t launch_band_empty(const BandArgs& a, void* out, float* lse, cudaStream_t stream) {
    const long long rows = band_rows(a);
    const cudaError_t e = cudaMemsetAsync(out, 0, static_cast<size_t>(rows) * a.D * (a.dtype == 0 ? 4 : 2), stream);
    if (e != cudaSuccess) return e;
    no_keys_kernel<<<static_cast<unsigned>((rows + 255) / 256), 256, 0, stream>>>(lse, rows);
    return cudaGetLastError();
}

size_t band_forward_workspace_bytes(const BandArgs& a) {
    return round256(a.dtype == 0 ? band_part_bytes(a, simt_splits(a)) : band_few_fits(a) ? band_few_part_bytes(a) : band_fwd_tc_part_bytes(a));
}

cudaError_t band_status(unsigned* status, bool reset) {
    unsigned fwd = 0, bwd = 0;
    cudaError_t e = band_fwd_status(&fwd, reset);
    if (e == cudaSuccess) e = band_bwd_status(&bwd, reset);
    *status = fwd | bwd;
    return e;
}

size_t band_backward_workspace_bytes(const BandArgs& a, bool want_bias) {
    return a.dtype == 0 ? band_simt_backward_workspace(a, want_bias) : band_bwd_tc_workspace(a, want_bias);
}

cudaError_t launch_band_forward(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    if (a.dtype == 0) return launch_band_simt_forward(a, out, lse, ws, stream);
    return band_few_fits(a) ? launch_band_few(a, out, lse, ws, stream) : launch_band_fwd_tc(a, out, lse, ws, stream);
}

cudaError_t launch_band_backward(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq,
                                 void* gk, void* gv, void* gbias, void* ws, cudaStream_t stream) {
    if (a.dtype != 0) return launch_band_bwd_tc(a, out, lse, gout, gq, gk, gv, gbias, ws, stream);
    return launch_band_simt_backward(a, out, lse, gout, gq, gk, gv, gbias, ws, stream);
}

}  // namespace dcn4
