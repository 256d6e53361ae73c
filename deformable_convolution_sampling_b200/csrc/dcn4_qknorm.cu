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
// Bound by HBM: x (and g) read once, out (or gx) written once.  A warp takes a few
// tokens (or some heads of one, where tokens are few) on its own: its lanes form the
// tokens' R / 2 angles, each once, into shared memory, and all heads use them.  A head is a group of lanes with two
// 16-byte pieces a lane, chosen so that both members of a pair are in one lane: the
// pieces p and p + R / 2 of the "halves" form (any two where pairs are neighbours), so
// that turning is arithmetic on registers; the sums are shuffles.  Only where R / 2 is
// no whole number of pieces does a head go through shared memory.
#include <algorithm>

#include "dcn4_band.cuh"
#include "dcn4_common.cuh"

namespace dcn4 {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr double kTwoPi = 6.283185307179586476925286766559, kInvTwoPi = 1.0 / kTwoPi;
constexpr int kMaxPairs = 128;  // D <= 256
// Which entries of a head make a pair, and where they are.
enum Mode { kNone, kHalves, kNeighbours, kExchange };

// How heads map to lanes and tokens to warps.
struct Shape {
    int lph;        // lanes of one head: a power of two
    int tokens;     // tokens of a unit; their pairs fit kMaxPairs
    int heads;      // heads of a unit's tokens: all of them, or a whole number of the warp's groups
    int chunks;     // units of the same tokens
    int apart;      // the pieces of a lane: p and p + apart for p < apart, neighbours behind 2 apart
    int mode;       // kExchange: the pairs of a lane's pieces do not match (shared memory)
    long long units;
    int grid;
};

__device__ __forceinline__ float group_sum(float v, int lph) {
    for (int o = lph >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A lane's two pieces as fp32.
template <typename T>
struct Lane {
    static constexpr int E = Elem<T>::per16;
    float f[2][E];
    __device__ __forceinline__ void from(const uint4 (&r)[2]) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float2 p[E / 2];
            unpack(r[c], p, T());
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                f[c][2 * e] = p[e].x;
                f[c][2 * e + 1] = p[e].y;
            }
        }
    }
    __device__ __forceinline__ void store(T* row, const int (&at)[2], int nchunk) const {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (at[c] >= nchunk) continue;
            float2 p[E / 2];
#pragma unroll
            for (int e = 0; e < E / 2; ++e) p[e] = make_float2(f[c][2 * e], f[c][2 * e + 1]);
            st_global(row + at[c] * E, pack(p, T()));
        }
    }
};

template <typename T>
__device__ __forceinline__ void load_pieces(uint4 (&r)[2], const T* row, const int (&at)[2], int nchunk) {
#pragma unroll
    for (int c = 0; c < 2; ++c) r[c] = at[c] < nchunk ? ld_stream(row + at[c] * Elem<T>::per16) : make_uint4(0u, 0u, 0u, 0u);
}

// What a warp knows of its lanes.
template <typename T, int MODE>
struct Warp {
    static constexpr int E = Elem<T>::per16;
    int lane, grp, hpw, nchunk, H;
    int at[2];       // the lane's pieces
    int pair;        // the lane's first pair, E from there on; -1: its pieces are not turned
    float2* cs;      // cos and sin of the tokens' pairs
    float* buf;      // D floats of this lane group (exchange)

    __device__ __forceinline__ Warp(const QkNormArgs& a, const Shape& sh, float* smem) {
        lane = threadIdx.x & 31;
        const int warp = threadIdx.x >> 5, p = lane & (sh.lph - 1);
        grp = lane / sh.lph;
        hpw = 32 / sh.lph;
        nchunk = a.D / E;
        H = a.Hq + a.Hk;
        const bool first = p < sh.apart;
        at[0] = first ? p : 2 * p;
        at[1] = first ? p + sh.apart : 2 * p + 1;
        pair = MODE == kNeighbours ? (at[0] * E < a.R ? p * E : -1) : first ? p * E : -1;
        cs = reinterpret_cast<float2*>(smem) + warp * kMaxPairs;
        buf = smem + kWarps * kMaxPairs * 2 + (warp * hpw + grp) * a.D;
    }
    // the angles of `count` tokens, each formed by one lane
    __device__ __forceinline__ void angles(const QkNormArgs& a, long long tok, int count) {
        if (MODE == kNone) return;
        const int h = a.R >> 1, per = a.axes == 2 ? h >> 1 : h;
        __syncwarp();  // the last unit's reads are done
        for (int e = lane; e < count * h; e += 32) {
            const int t = e / h, i = e - t * h;
            const float pos = __ldg(a.pos + (tok + t) * a.axes + (i >= per ? 1 : 0));
            double f = static_cast<double>(pos) * static_cast<double>(__ldg(a.inv_freq + i));
            f -= kTwoPi * rint(f * kInvTwoPi);
            float s, c;
            sincosf(static_cast<float>(f), &s, &c);
            cs[e] = make_float2(c, s);
        }
        __syncwarp();
    }
    // Turns a head's pairs by the angles of token t of the unit (dir = 1) or back (dir = -1).
    __device__ __forceinline__ void turn(Lane<T>& x, const QkNormArgs& a, int t, float dir) {
        if (MODE == kNone) return;
        const int h = a.R >> 1;
        const float2* q = cs + t * h;
        if (MODE != kExchange) {
            if (pair < 0) return;
            q += pair;
            // halves: pair e of the lane is (f[0][e], f[1][e]); neighbours: (f[c][2 e], f[c][2 e + 1]) of piece c,
            // of which some may lie beyond R
            const int here = MODE == kNeighbours ? h - pair : E;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (MODE == kNeighbours && e >= here) break;
                float &u = MODE == kHalves ? x.f[0][e] : x.f[e / (E / 2)][2 * (e % (E / 2))],
                      &v = MODE == kHalves ? x.f[1][e] : x.f[e / (E / 2)][2 * (e % (E / 2)) + 1];
                const float2 r = q[e];
                const float s = r.y * dir, w = u;
                u = w * r.x - v * s;
                v = v * r.x + w * s;
            }
            return;
        }
        __syncwarp();  // the previous head's reads of buf are done
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (at[c] < nchunk)
#pragma unroll
                for (int e = 0; e < E; ++e) buf[at[c] * E + e] = x.f[c][e];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = at[c] * E + e;
                if (d < a.R) {
                    const bool lo = d < h;
                    const float2 r = q[lo ? d : d - h];
                    const float s = r.y * dir, o = buf[lo ? d + h : d - h];
                    x.f[c][e] = lo ? x.f[c][e] * r.x - o * s : x.f[c][e] * r.x + o * s;
                }
            }
    }
};

// A unit's heads of one side (queries or keys): `count` tokens from tok on, heads [h0, h0 + heads) of H.
template <typename T>
struct Side {
    const T* x;
    long long batch, row;
    int H, h0, heads;
    __device__ __forceinline__ Side(const QkNormArgs& a, int side, int lo, int hi) {
        x = static_cast<const T*>(side ? a.k : a.q);
        batch = side ? a.k_batch : a.q_batch;
        row = side ? a.k_row : a.q_row;
        H = side ? a.Hk : a.Hq;
        h0 = max(lo - (side ? a.Hq : 0), 0);
        heads = max(min(hi - (side ? a.Hq : 0), H) - h0, 0);
    }
    // item `it` of the unit: its token, and where its head lies in the input and in a dense tensor
    __device__ __forceinline__ void place(const QkNormArgs& a, long long tok, int it, int& t, long long& in, long long& dense, int D) const {
        t = it / heads;
        const int h = h0 + it - t * heads;
        const long long at = tok + t, n = at / a.L;
        in = n * batch + (at - n * a.L) * row + static_cast<long long>(h) * D;
        dense = (at * H + h) * D;
    }
};

template <typename T>
__device__ __forceinline__ void load_weight(Lane<T>& w, const void* p, const int (&at)[2], int nchunk) {
    if (p) {
        uint4 r[2];
        load_pieces<T>(r, static_cast<const T*>(p), at, nchunk);
        w.from(r);
    } else {
#pragma unroll
        for (int e = 0; e < 2 * Elem<T>::per16; ++e) w.f[e / Elem<T>::per16][e % Elem<T>::per16] = 1.f;
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 6) qknorm_forward_kernel(QkNormArgs a, Shape sh, T* __restrict__ qo, T* __restrict__ ko) {
    constexpr int E = Elem<T>::per16;
    extern __shared__ __align__(16) float qk_smem[];
    Warp<T, MODE> wp(a, sh, qk_smem);
    const long long total = static_cast<long long>(a.N) * a.L;
    for (long long u = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5); u < sh.units; u += static_cast<long long>(gridDim.x) * kWarps) {
        const long long tok = u / sh.chunks * sh.tokens;
        const int count = static_cast<int>(total - tok < sh.tokens ? total - tok : sh.tokens);
        const int lo = static_cast<int>(u % sh.chunks) * sh.heads;
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const Side<T> sd(a, side, lo, lo + sh.heads);
            const int items = count * sd.heads;
            if (items) {
                uint4 raw[2];
                long long dense;
                int t;
                auto fetch = [&](int it) {
                    long long in;
                    sd.place(a, tok, min(it, items - 1), t, in, dense, a.D);
                    load_pieces<T>(raw, sd.x + in, wp.at, it < items ? wp.nchunk : 0);
                };
                fetch(wp.grp);
                Lane<T> w;
                load_weight<T>(w, side ? a.wk : a.wq, wp.at, wp.nchunk);
                if (side == 0 || lo >= a.Hq) wp.angles(a, tok, count);
                T* out = side ? ko : qo;
                for (int at = 0; at < items; at += wp.hpw) {  // whole warps: the lanes shuffle
                    Lane<T> x;
                    x.from(raw);
                    const long long to = dense;
                    const int tx = t;
                    if (at + wp.hpw < items) fetch(at + wp.hpw + wp.grp);
                    float ss = 0.f;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E; ++e) ss = fmaf(x.f[c][e], x.f[c][e], ss);
                    const float s = rsqrtf(group_sum(ss, sh.lph) / a.D + a.eps);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E; ++e) x.f[c][e] = x.f[c][e] * s * w.f[c][e];
                    wp.turn(x, a, tx, 1.f);
                    if (at + wp.grp < items) x.store(out + to, wp.at, wp.nchunk);
                }
            }
        }
    }
}

// gx, and this CTA's sums of gw: part[cta][2][D] (queries, keys).
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 4)
    qknorm_backward_kernel(QkNormArgs a, Shape sh, const T* __restrict__ gqo, const T* __restrict__ gko,
                           T* __restrict__ gq, T* __restrict__ gk, float* __restrict__ part) {
    constexpr int E = Elem<T>::per16;
    extern __shared__ __align__(16) float qk_smem[];
    Warp<T, MODE> wp(a, sh, qk_smem);
    const long long total = static_cast<long long>(a.N) * a.L;
    float acc[2][2][E] = {};  // queries' and keys' sums of the lane's entries
    for (long long u = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5); u < sh.units; u += static_cast<long long>(gridDim.x) * kWarps) {
        const long long tok = u / sh.chunks * sh.tokens;
        const int count = static_cast<int>(total - tok < sh.tokens ? total - tok : sh.tokens);
        const int lo = static_cast<int>(u % sh.chunks) * sh.heads;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const Side<T> sd(a, side, lo, lo + sh.heads);
            const int items = count * sd.heads;
            if (items) {
                uint4 raw_x[2], raw_g[2];
                long long dense;
                int t;
                auto fetch = [&](int it) {
                    long long in;
                    sd.place(a, tok, min(it, items - 1), t, in, dense, a.D);
                    const int pieces = it < items ? wp.nchunk : 0;
                    load_pieces<T>(raw_x, sd.x + in, wp.at, pieces);
                    load_pieces<T>(raw_g, (side ? gko : gqo) + dense, wp.at, pieces);
                };
                fetch(wp.grp);
                Lane<T> w;
                load_weight<T>(w, side ? a.wk : a.wq, wp.at, wp.nchunk);
                if (side == 0 || lo >= a.Hq) wp.angles(a, tok, count);
                for (int at = 0; at < items; at += wp.hpw) {
                    Lane<T> x, g;
                    x.from(raw_x);
                    g.from(raw_g);
                    const long long to = dense;
                    const int tx = t;
                    if (at + wp.hpw < items) fetch(at + wp.hpw + wp.grp);
                    wp.turn(g, a, tx, -1.f);
                    float ss = 0.f, gx = 0.f;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            ss = fmaf(x.f[c][e], x.f[c][e], ss);
                            gx = fmaf(g.f[c][e] * w.f[c][e], x.f[c][e], gx);
                        }
                    ss = group_sum(ss, sh.lph);
                    gx = group_sum(gx, sh.lph);
                    const float s = rsqrtf(ss / a.D + a.eps), back = s * s * (gx / a.D);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E; ++e) {  // (a head past the last has x = g = 0)
                            acc[side][c][e] = fmaf(g.f[c][e], x.f[c][e] * s, acc[side][c][e]);
                            x.f[c][e] = s * (g.f[c][e] * w.f[c][e] - x.f[c][e] * back);
                        }
                    if (at + wp.grp < items) x.store((side ? gk : gq) + to, wp.at, wp.nchunk);
                }
            }
        }
    }
    // the CTA's sums: lane groups and warps in a fixed order
    if (!part) return;
    float* bufs = qk_smem + kWarps * kMaxPairs * 2;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (wp.at[c] < wp.nchunk)
#pragma unroll
                for (int e = 0; e < E; ++e) wp.buf[wp.at[c] * E + e] = acc[side][c][e];
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += kThreads) {
            float s = 0.f;
            for (int w = 0; w < kWarps * wp.hpw; ++w) s += bufs[w * a.D + d];
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
    s.mode = !a.R ? kNone : a.interleaved ? kNeighbours : (a.R / 2) % elems ? kExchange : kHalves;
    s.apart = s.mode == kHalves ? a.R / 2 / elems : 0;
    // lanes: one for each pair of matching pieces, one for each two of the rest
    const int lanes = s.apart + (nchunk - 2 * s.apart + 1) / 2;
    s.lph = 1;
    while (s.lph < lanes) s.lph *= 2;
    const int hpw = 32 / s.lph;
    const long long total = static_cast<long long>(a.N) * a.L, busy = 24LL * kBandSms;  // warps that hide the loads
    // some sixteen steps of a warp a unit, fewer while that leaves SMs without their warps: then a token's
    // heads are split, too
    s.tokens = static_cast<int>(std::max<long long>(1, std::min<long long>(16LL * hpw / H, total / busy)));
    if (a.R) s.tokens = std::min(s.tokens, kMaxPairs / (a.R / 2));
    const long long sets = (total + s.tokens - 1) / s.tokens;
    const int groups = (H + hpw - 1) / hpw;
    s.chunks = static_cast<int>(std::max<long long>(1, std::min<long long>(groups, (busy + sets - 1) / std::max<long long>(sets, 1))));
    s.heads = s.chunks == 1 ? H : (groups + s.chunks - 1) / s.chunks * hpw;
    s.chunks = (H + s.heads - 1) / s.heads;
    s.units = sets * s.chunks;
    s.grid = static_cast<int>(std::min<long long>((s.units + kWarps - 1) / kWarps, 8LL * kBandSms));
    return s;
}

size_t smem_bytes(const QkNormArgs& a, const Shape& s) {
    return (static_cast<size_t>(kWarps) * kMaxPairs * 2 + static_cast<size_t>(kWarps) * (32 / s.lph) * a.D) * sizeof(float);
}

template <typename T>
cudaError_t forward_typed(const QkNormArgs& a, void* qo, void* ko, cudaStream_t stream) {
    const Shape s = shape_of(a, Elem<T>::per16);
    const auto kernel = s.mode == kNone ? qknorm_forward_kernel<T, kNone> : s.mode == kHalves ? qknorm_forward_kernel<T, kHalves>
                        : s.mode == kNeighbours ? qknorm_forward_kernel<T, kNeighbours> : qknorm_forward_kernel<T, kExchange>;
    kernel<<<s.grid, kThreads, smem_bytes(a, s), stream>>>(a, s, static_cast<T*>(qo), static_cast<T*>(ko));
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(const QkNormArgs& a, const void* gqo, const void* gko, void* gq, void* gk, void* gwq,
                           void* gwk, void* ws, cudaStream_t stream) {
    const Shape s = shape_of(a, Elem<T>::per16);
    float* part = (gwq || gwk) ? static_cast<float*>(ws) : nullptr;
    const auto kernel = s.mode == kNone ? qknorm_backward_kernel<T, kNone> : s.mode == kHalves ? qknorm_backward_kernel<T, kHalves>
                        : s.mode == kNeighbours ? qknorm_backward_kernel<T, kNeighbours> : qknorm_backward_kernel<T, kExchange>;
    kernel<<<s.grid, kThreads, smem_bytes(a, s), stream>>>(a, s, static_cast<const T*>(gqo), static_cast<const T*>(gko),
                                                          static_cast<T*>(gq), static_cast<T*>(gk), part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !part) return e;
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
