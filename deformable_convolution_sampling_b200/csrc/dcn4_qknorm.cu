// dcn4_qknorm.cu — RMS norm of every query and key head and the position
// rotation, in one pass over q and k, and its backward.
//
// With x a head's D entries, s = 1 / sqrt(mean(x^2) + eps), y = s x w, and
// (a, b) a pair of the first R entries of y at angle f = pos * inv_freq:
//     out = (a cos f - b sin f, a sin f + b cos f)
// and backwards, with g the upstream gradient turned back by -f,
//     gw = sum g s x,     gx = s (g w - x s^2 mean(g w x)).
// The angle is formed and reduced to [-pi, pi] in 64 bits (a position of 10^5
// times a frequency of 1 leaves 2^-7 of a radian in 32 bits), once per token
// and pair into shared memory; all heads of the token use it.  Everything else
// is 32 bits, rounded once.
//
// Bound by HBM: x (and g) read once, out (or gx) written once.  A head is a
// group of lanes of one warp with 16 bytes a lane, so loads and stores are
// whole sectors and the sums are shuffles; pairs of the "halves" form, whose
// members sit in different lanes, are exchanged through shared memory.
#include <algorithm>

#include "dcn4_band.cuh"
#include "dcn4_common.cuh"

namespace dcn4 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTokens = 32;  // tokens of one CTA's step at most
constexpr double kTwoPi = 6.283185307179586476925286766559, kInvTwoPi = 1.0 / kTwoPi;

// How heads map to lanes and tokens to CTAs.
struct Shape {
    int lph;     // lanes of one head: a power of two
    int tokens;  // tokens of one step
    long long steps;
    int grid;
};

__device__ __forceinline__ float group_sum(float v, int lph) {
    for (int o = lph >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, int CPL>
struct Lane {  // a lane's CPL chunks of 16 bytes as fp32
    static constexpr int E = Elem<T>::per16;
    float f[CPL * E];
};

template <typename T, int CPL>
__device__ __forceinline__ void load_lane(Lane<T, CPL>& x, const T* row, int gl, int lph, int nchunk) {
    constexpr int E = Elem<T>::per16;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int ch = gl + c * lph;
        float2 p[E / 2];
        const uint4 r = ch < nchunk ? ld_stream(row + ch * E) : make_uint4(0u, 0u, 0u, 0u);
        unpack(r, p, T());
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            x.f[c * E + 2 * e] = p[e].x;
            x.f[c * E + 2 * e + 1] = p[e].y;
        }
    }
}
template <typename T, int CPL>
__device__ __forceinline__ void store_lane(const Lane<T, CPL>& x, T* row, int gl, int lph, int nchunk) {
    constexpr int E = Elem<T>::per16;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int ch = gl + c * lph;
        if (ch >= nchunk) continue;
        float2 p[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) p[e] = make_float2(x.f[c * E + 2 * e], x.f[c * E + 2 * e + 1]);
        st_global(row + ch * E, pack(p, T()));
    }
}

// Turns the pairs of a head by the angles cs (dir = 1) or back (dir = -1).
// buf: this lane group's D floats of shared memory, for the halves form.
template <typename T, int CPL>
__device__ __forceinline__ void turn(Lane<T, CPL>& x, const float2* cs, float* buf, int R, int interleaved, float dir,
                                     int gl, int lph, int nchunk) {
    constexpr int E = Elem<T>::per16;
    if (R == 0) return;
    if (interleaved) {
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const int d0 = (gl + c * lph) * E;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                if (d0 + e < R) {
                    const float2 t = cs[(d0 + e) >> 1];
                    const float s = t.y * dir, a = x.f[c * E + e], b = x.f[c * E + e + 1];
                    x.f[c * E + e] = a * t.x - b * s;
                    x.f[c * E + e + 1] = b * t.x + a * s;
                }
        }
        return;
    }
    const int h = R >> 1;
    __syncwarp();  // the previous head's reads of buf are done
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int ch = gl + c * lph;
        if (ch < nchunk) {
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *reinterpret_cast<float4*>(buf + ch * E + e) =
                    make_float4(x.f[c * E + e], x.f[c * E + e + 1], x.f[c * E + e + 2], x.f[c * E + e + 3]);
        }
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int d0 = (gl + c * lph) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = d0 + e;
            if (d < R) {
                const bool lo = d < h;
                const float2 t = cs[lo ? d : d - h];
                const float s = t.y * dir, o = buf[lo ? d + h : d - h];
                x.f[c * E + e] = lo ? x.f[c * E + e] * t.x - o * s : x.f[c * E + e] * t.x + o * s;
            }
        }
    }
}

// cos and sin of every (token of the step, pair).
__device__ __forceinline__ void angles(const QkNormArgs& a, float2* cs, long long tok0, int ntok) {
    const int h = a.R >> 1, per = a.axes == 2 ? h >> 1 : h;
    for (int i = threadIdx.x; i < ntok * h; i += kThreads) {
        const int t = i / h, pr = i - t * h;
        const float pos = a.pos[(tok0 + t) * a.axes + (pr >= per ? 1 : 0)];
        double f = static_cast<double>(pos) * static_cast<double>(a.inv_freq[pr]);
        f -= kTwoPi * rint(f * kInvTwoPi);
        float s, c;
        sincosf(static_cast<float>(f), &s, &c);
        cs[i] = make_float2(c, s);
    }
}

template <typename T, int CPL>
__device__ __forceinline__ void load_weight(Lane<T, CPL>& w, const void* p, int gl, int lph, int nchunk) {
    if (p) {
        load_lane<T, CPL>(w, static_cast<const T*>(p), gl, lph, nchunk);
    } else {
#pragma unroll
        for (int e = 0; e < CPL * Elem<T>::per16; ++e) w.f[e] = 1.f;
    }
}

template <typename T, int CPL>
__global__ void __launch_bounds__(kThreads) qknorm_forward_kernel(QkNormArgs a, Shape sh, T* __restrict__ qo, T* __restrict__ ko) {
    constexpr int E = Elem<T>::per16;
    extern __shared__ __align__(16) float qk_smem[];
    float2* cs = reinterpret_cast<float2*>(qk_smem);              // [tokens][R / 2]
    float* bufs = qk_smem + sh.tokens * a.R + ((sh.tokens * a.R) & 3 ? 4 - ((sh.tokens * a.R) & 3) : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lph = sh.lph, gl = lane & (lph - 1), grp = lane / lph, hpw = 32 / lph;
    const int nchunk = a.D / E, H = a.Hq + a.Hk;
    float* buf = bufs + (warp * hpw + grp) * a.D;
    Lane<T, CPL> wq, wk;
    load_weight<T, CPL>(wq, a.wq, gl, lph, nchunk);
    load_weight<T, CPL>(wk, a.wk, gl, lph, nchunk);
    const long long total = static_cast<long long>(a.N) * a.L;
    for (long long st = blockIdx.x; st < sh.steps; st += gridDim.x) {
        const long long tok0 = st * sh.tokens;
        const int ntok = static_cast<int>(total - tok0 < sh.tokens ? total - tok0 : sh.tokens);
        if (a.R) {
            __syncthreads();
            angles(a, cs, tok0, ntok);
            __syncthreads();
        }
        const int items = ntok * H;
        for (int it0 = warp * hpw; it0 < items; it0 += kWarps * hpw) {  // whole warps: the lanes shuffle
            const int it = it0 + grp;
            const bool on = it < items;
            const int t = on ? it / H : 0, h = on ? it - t * H : 0;
            const bool isq = h < a.Hq;
            const int hh = isq ? h : h - a.Hq;
            const long long tok = tok0 + t, n = tok / a.L, l = tok - n * a.L;
            const T* row = isq ? static_cast<const T*>(a.q) + n * a.q_batch + l * a.q_row
                               : static_cast<const T*>(a.k) + n * a.k_batch + l * a.k_row;
            Lane<T, CPL> x;
            load_lane<T, CPL>(x, row + static_cast<long long>(hh) * a.D, gl, lph, on ? nchunk : 0);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < CPL * E; ++e) ss = fmaf(x.f[e], x.f[e], ss);
            const float s = rsqrtf(group_sum(ss, lph) / a.D + a.eps);
#pragma unroll
            for (int e = 0; e < CPL * E; ++e) x.f[e] = x.f[e] * s * (isq ? wq.f[e] : wk.f[e]);
            turn<T, CPL>(x, cs + t * (a.R >> 1), buf, a.R, a.interleaved, 1.f, gl, lph, nchunk);
            T* out = isq ? qo + (tok * a.Hq + hh) * a.D : ko + (tok * a.Hk + hh) * a.D;
            store_lane<T, CPL>(x, out, gl, lph, on ? nchunk : 0);
        }
    }
}

// gx, and this CTA's sums of gw: part[cta][2][D] (queries, keys).
template <typename T, int CPL>
__global__ void __launch_bounds__(kThreads)
    qknorm_backward_kernel(QkNormArgs a, Shape sh, const T* __restrict__ gqo, const T* __restrict__ gko,
                           T* __restrict__ gq, T* __restrict__ gk, float* __restrict__ part) {
    constexpr int E = Elem<T>::per16;
    extern __shared__ __align__(16) float qk_smem[];
    float2* cs = reinterpret_cast<float2*>(qk_smem);
    float* bufs = qk_smem + sh.tokens * a.R + ((sh.tokens * a.R) & 3 ? 4 - ((sh.tokens * a.R) & 3) : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lph = sh.lph, gl = lane & (lph - 1), grp = lane / lph, hpw = 32 / lph;
    const int nchunk = a.D / E, H = a.Hq + a.Hk;
    float* buf = bufs + (warp * hpw + grp) * a.D;
    Lane<T, CPL> wq, wk, aq, ak;
    load_weight<T, CPL>(wq, a.wq, gl, lph, nchunk);
    load_weight<T, CPL>(wk, a.wk, gl, lph, nchunk);
#pragma unroll
    for (int e = 0; e < CPL * E; ++e) aq.f[e] = ak.f[e] = 0.f;
    const long long total = static_cast<long long>(a.N) * a.L;
    for (long long st = blockIdx.x; st < sh.steps; st += gridDim.x) {
        const long long tok0 = st * sh.tokens;
        const int ntok = static_cast<int>(total - tok0 < sh.tokens ? total - tok0 : sh.tokens);
        if (a.R) {
            __syncthreads();
            angles(a, cs, tok0, ntok);
            __syncthreads();
        }
        const int items = ntok * H;
        for (int it0 = warp * hpw; it0 < items; it0 += kWarps * hpw) {
            const int it = it0 + grp;
            const bool on = it < items;
            const int t = on ? it / H : 0, h = on ? it - t * H : 0;
            const bool isq = h < a.Hq;
            const int hh = isq ? h : h - a.Hq;
            const long long tok = tok0 + t, n = tok / a.L, l = tok - n * a.L;
            const T* row = isq ? static_cast<const T*>(a.q) + n * a.q_batch + l * a.q_row
                               : static_cast<const T*>(a.k) + n * a.k_batch + l * a.k_row;
            const long long dense = isq ? (tok * a.Hq + hh) * a.D : (tok * a.Hk + hh) * a.D;
            Lane<T, CPL> x, g;
            load_lane<T, CPL>(x, row + static_cast<long long>(hh) * a.D, gl, lph, on ? nchunk : 0);
            load_lane<T, CPL>(g, (isq ? gqo : gko) + dense, gl, lph, on ? nchunk : 0);
            turn<T, CPL>(g, cs + t * (a.R >> 1), buf, a.R, a.interleaved, -1.f, gl, lph, nchunk);
            float ss = 0.f, gx = 0.f;
#pragma unroll
            for (int e = 0; e < CPL * E; ++e) {
                ss = fmaf(x.f[e], x.f[e], ss);
                gx = fmaf(g.f[e] * (isq ? wq.f[e] : wk.f[e]), x.f[e], gx);
            }
            ss = group_sum(ss, lph);
            gx = group_sum(gx, lph);
            const float s = rsqrtf(ss / a.D + a.eps), back = s * s * (gx / a.D);
#pragma unroll
            for (int e = 0; e < CPL * E; ++e) {
                const float gw = on ? g.f[e] * (x.f[e] * s) : 0.f;
                const float w = isq ? wq.f[e] : wk.f[e];
                if (isq) aq.f[e] += gw; else ak.f[e] += gw;
                x.f[e] = s * (g.f[e] * w - x.f[e] * back);
            }
            store_lane<T, CPL>(x, (isq ? gq : gk) + dense, gl, lph, on ? nchunk : 0);
        }
    }
    // the CTA's sums: lane groups and warps in a fixed order
    if (!part) return;
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            if (gl + c * lph < nchunk)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    buf[(gl + c * lph) * E + e] = side ? ak.f[c * E + e] : aq.f[c * E + e];
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += kThreads) {
            float s = 0.f;
            for (int w = 0; w < kWarps * hpw; ++w) s += bufs[w * a.D + d];
            part[(static_cast<long long>(blockIdx.x) * 2 + side) * a.D + d] = s;
        }
    }
}

// gw[d] = the sum of the CTAs' parts: a warp per entry.
template <typename T>
__global__ void __launch_bounds__(kThreads) qknorm_weights_kernel(const float* __restrict__ part, int ctas, int D,
                                                                  T* __restrict__ gwq, T* __restrict__ gwk) {
    const int e = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= 2 * D) return;
    float s = 0.f;
    for (int c = lane; c < ctas; c += 32) s += part[static_cast<long long>(c) * 2 * D + e];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    T* to = e < D ? gwq : gwk;
    if (lane == 0 && to) to[e < D ? e : e - D] = from_f32<T>(s);
}

Shape shape_of(const QkNormArgs& a, int elems) {
    Shape s;
    const int nchunk = a.D / elems, H = a.Hq + a.Hk;
    s.lph = 1;
    while (s.lph < nchunk && s.lph < 32) s.lph *= 2;
    const long long total = static_cast<long long>(a.N) * a.L;
    // four heads a warp's lane group and step, fewer tokens while that leaves SMs without a CTA
    long long t = 4LL * kWarps * (32 / s.lph) / H;
    t = std::min<long long>(std::max<long long>(t, 1), kMaxTokens);
    while (t > 1 && (total + t - 1) / t < 2 * kBandSms) t /= 2;
    s.tokens = static_cast<int>(t);
    s.steps = (total + t - 1) / t;
    s.grid = static_cast<int>(std::min<long long>(s.steps, 8LL * kBandSms));
    return s;
}

template <typename T>
size_t smem_bytes(const QkNormArgs& a, const Shape& s) {
    return (static_cast<size_t>(s.tokens) * a.R + 4 + static_cast<size_t>(kWarps) * (32 / s.lph) * a.D) * sizeof(float);
}

template <typename T>
cudaError_t forward_typed(const QkNormArgs& a, void* qo, void* ko, cudaStream_t stream) {
    const Shape s = shape_of(a, Elem<T>::per16);
    const size_t smem = smem_bytes<T>(a, s);
    if (a.D / Elem<T>::per16 > 32)
        qknorm_forward_kernel<T, 2><<<s.grid, kThreads, smem, stream>>>(a, s, static_cast<T*>(qo), static_cast<T*>(ko));
    else
        qknorm_forward_kernel<T, 1><<<s.grid, kThreads, smem, stream>>>(a, s, static_cast<T*>(qo), static_cast<T*>(ko));
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(const QkNormArgs& a, const void* gqo, const void* gko, void* gq, void* gk, void* gwq,
                           void* gwk, void* ws, cudaStream_t stream) {
    const Shape s = shape_of(a, Elem<T>::per16);
    const size_t smem = smem_bytes<T>(a, s);
    float* part = (gwq || gwk) ? static_cast<float*>(ws) : nullptr;
    const T *uq = static_cast<const T*>(gqo), *uk = static_cast<const T*>(gko);
    T *oq = static_cast<T*>(gq), *ok = static_cast<T*>(gk);
    if (s.grid > 0) {
        if (a.D / Elem<T>::per16 > 32)
            qknorm_backward_kernel<T, 2><<<s.grid, kThreads, smem, stream>>>(a, s, uq, uk, oq, ok, part);
        else
            qknorm_backward_kernel<T, 1><<<s.grid, kThreads, smem, stream>>>(a, s, uq, uk, oq, ok, part);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!part) return cudaSuccess;
    qknorm_weights_kernel<T><<<(2 * a.D + kWarps - 1) / kWarps, kThreads, 0, stream>>>(
        part, s.grid, a.D, static_cast<T*>(gwq), static_cast<T*>(gwk));
    return cudaGetLastError();
}

}  // namespace

size_t qknorm_backward_workspace_bytes(const QkNormArgs& a) {
    const Shape s = shape_of(a, a.dtype == 0 ? 4 : 8);
    return (static_cast<size_t>(s.grid) * 2 * a.D * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_qknorm_forward(const QkNormArgs& a, void* qo, void* ko, cudaStream_t stream) {
    switch (a.dtype) {
        case 0: return forward_typed<float>(a, qo, ko, stream);
        case 1: return forward_typed<__half>(a, qo, ko, stream);
        case 2: return forward_typed<__nv_bfloat16>(a, qo, ko, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_qknorm_backward(const QkNormArgs& a, const void* gqo, const void* gko, void* gq, void* gk,
                                   void* gwq, void* gwk, void* ws, cudaStream_t stream) {
    switch (a.dtype) {
        case 0: return backward_typed<float>(a, gqo, gko, gq, gk, gwq, gwk, ws, stream);
        case 1: return backward_typed<__half>(a, gqo, gko, gq, gk, gwq, gwk, ws, stream);
        case 2: return backward_typed<__nv_bfloat16>(a, gqo, gko, gq, gk, gwq, gwk, ws, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace dcn4
