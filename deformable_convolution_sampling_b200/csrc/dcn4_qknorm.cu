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
// and pair into shared memory; all heads of the token use it.  Its sine and cosine
// are those of its 32 leading bits and a first-order term of the rest.  Everything
// else is 32 bits, rounded once.
//
// Bound by HBM: x (and g) read once, out (or gx) written once.  A warp takes a few
// tokens (or some heads of one, where tokens are few) on its own: its lanes form the
// tokens' R / 2 angles, each once, into shared memory, and all heads use them.  A head is a group of lanes with two
// 16-byte pieces a lane, chosen so that both members of a pair are in one lane: the
// pieces p and p + R / 2 of the "halves" form (any two where pairs are neighbours), so
// that turning is arithmetic on registers; the sums are shuffles.  Only where R / 2 is
// no whole number of pieces does a head go through shared memory.  4 x 4096 tokens, 20
// heads of 128, bf16: 42 us forward (4.0 TB/s; a copy takes 28), 67 us backward, 3 the
// weights' sums.  Few loads are in flight (20 and 12 warps an SM, one item each).
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
// CTAs an SM.  The 16-bit forwards spill a little at 5 (24 bytes where pairs are halves, 56
// through shared memory), the backwards at 3 only there (16).  At 6 and 4 they spill more,
// and uneven shares of the tokens cost a round: 46 and 77 us for 4 x 4096 tokens of 20 heads
// of 128.
constexpr int kForwardCtas = 5, kBackwardCtas = 3;

// The units of a warp: all heads of a run of tokens, every warp's as long as the next
// one's, or, where tokens are few, some heads of one token at a time.
struct Units {
    long long at, end, step;
    __device__ __forceinline__ Units(const Shape& sh, long long total) {
        const long long w = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5), all = static_cast<long long>(gridDim.x) * kWarps;
        const bool run = sh.chunks == 1;
        at = run ? total * w / all : w;
        end = run ? total * (w + 1) / all : sh.units;
        step = run ? sh.tokens : all;
    }
};

__device__ __forceinline__ float group_sum(float v, int lph) {
    for (int o = lph >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Two fp32 values handled by one instruction.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ float2 unf2(F2 v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A lane's two pieces as pairs of fp32.
template <typename T>
struct Lane {
    static constexpr int P = Elem<T>::per16 / 2;
    F2 f[2][P];
    __device__ __forceinline__ void from(const uint4 (&r)[2]) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float2 p[P];
            unpack(r[c], p, T());
#pragma unroll
            for (int e = 0; e < P; ++e) f[c][e] = f2(p[e].x, p[e].y);
        }
    }
    __device__ __forceinline__ void store(T* row, const int (&at)[2], int nchunk) const {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (at[c] >= nchunk) continue;
            float2 p[P];
#pragma unroll
            for (int e = 0; e < P; ++e) p[e] = unf2(f[c][e]);
            st_global(row + at[c] * 2 * P, pack(p, T()));
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
    float *cs, *sn;  // cos and sin of the tokens' pairs
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
        cs = smem + warp * 2 * kMaxPairs;
        sn = cs + kMaxPairs;
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
            // 32 bits of an angle near pi leave up to 2^-23 of it: the rest turns sin and cos to first order
            const float lead = static_cast<float>(f), rest = static_cast<float>(f - lead);
            float sine, cosine;
            sincosf(lead, &sine, &cosine);
            sn[e] = fmaf(cosine, rest, sine);
            cs[e] = fmaf(-sine, rest, cosine);
        }
        __syncwarp();
    }
    // Turns a head's pairs by the angles of token t of the unit (dir = 1) or back (dir = -1).
    __device__ __forceinline__ void turn(Lane<T>& x, const QkNormArgs& a, int t, float dir) {
        if (MODE == kNone) return;
        const int h = a.R >> 1;
        const float *c = cs + t * h, *n = sn + t * h;
        if (MODE == kHalves) {
            if (pair < 0) return;
#pragma unroll
            for (int e = 0; e < E / 2; e += 2) {  // four pairs: h is a multiple of E here
                const float4 c4 = *reinterpret_cast<const float4*>(c + pair + 2 * e), n4 = *reinterpret_cast<const float4*>(n + pair + 2 * e);
                const F2 cc[2] = {f2(c4.x, c4.y), f2(c4.z, c4.w)};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float sx = (k ? n4.z : n4.x) * dir, sy = (k ? n4.w : n4.y) * dir;
                    const F2 u = x.f[0][e + k], v = x.f[1][e + k];
                    x.f[0][e + k] = fma2(v, f2(-sx, -sy), mul2(u, cc[k]));
                    x.f[1][e + k] = fma2(u, f2(sx, sy), mul2(v, cc[k]));
                }
            }
        } else if (MODE == kNeighbours) {
            if (pair < 0) return;
#pragma unroll
            for (int e = 0; e < E; ++e) {  // of the lane's pairs some may lie beyond R
                if (pair + e >= h) break;
                F2& v = x.f[e / (E / 2)][e % (E / 2)];
                const float2 p = unf2(v);
                const float ce = c[pair + e], se = n[pair + e] * dir;
                v = f2(p.x * ce - p.y * se, p.y * ce + p.x * se);
            }
        } else {
            __syncwarp();  // the previous head's reads of buf are done
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (at[k] < nchunk)
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) *reinterpret_cast<float2*>(buf + at[k] * E + 2 * e) = unf2(x.f[k][e]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const int d = at[k] * E + 2 * e;
                    float2 v = unf2(x.f[k][e]);
                    auto one = [&](float w, int d) {
                        if (d >= a.R) return w;
                        const bool lo = d < h;
                        const int i = lo ? d : d - h;
                        const float s = n[i] * dir, o = buf[lo ? d + h : d - h];
                        return lo ? w * c[i] - o * s : w * c[i] + o * s;
                    };
                    v.x = one(v.x, d);
                    v.y = one(v.y, d + 1);
                    x.f[k][e] = f2(v.x, v.y);
                }
        }
    }
};

// Where a lane group is among a unit's heads of one side (queries or keys): tokens
// from tok = (n, l) on, `heads` heads of each from h0 on.  It goes on by the warp's
// groups with additions only (a division an item cost more than its arithmetic).
struct Walk {
    int heads, t, h, dt, dh;
    __device__ __forceinline__ Walk(int heads, int grp, int hpw) : heads(heads) {
        t = grp / heads;
        h = grp - t * heads;
        dt = hpw / heads;
        dh = hpw - dt * heads;
    }
    __device__ __forceinline__ void next() {
        t += dt;
        h += dh;
        if (h >= heads) h -= heads, ++t;
    }
};
// Elements from token (n, l) on to the token t behind it.
__device__ __forceinline__ long long ahead(int L, int l, int t, long long batch, long long row) {
    if (l + t < L) return t * row;
    const int at = l + t;
    return at / L * batch + (at % L - l) * row;
}

// A lane's pieces of a weight, as they are stored; NULL: ones.
template <typename T>
__device__ __forceinline__ void load_weight(uint4 (&w)[2], const void* p, const int (&at)[2], int nchunk) {
    if (p) {
        load_pieces<T>(w, static_cast<const T*>(p), at, nchunk);
    } else {
        float2 one[Elem<T>::per16 / 2];
#pragma unroll
        for (int e = 0; e < Elem<T>::per16 / 2; ++e) one[e] = make_float2(1.f, 1.f);
        w[0] = w[1] = pack(one, T());
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, kForwardCtas) qknorm_forward_kernel(QkNormArgs a, Shape sh, T* __restrict__ qo, T* __restrict__ ko) {
    constexpr int E = Elem<T>::per16;
    extern __shared__ __align__(16) float qk_smem[];
    Warp<T, MODE> wp(a, sh, qk_smem);
    const long long total = static_cast<long long>(a.N) * a.L;
    const float inv_d = 1.f / a.D;
    const Units un(sh, total);
    for (long long u = un.at; u < un.end; u += un.step) {
        const bool run = sh.chunks == 1;
        const long long tok = run ? u : u / sh.chunks;
        const int count = run ? static_cast<int>(un.end - u < sh.tokens ? un.end - u : sh.tokens) : 1;
        const int lo = run ? 0 : static_cast<int>(u % sh.chunks) * sh.heads;
        const long long n = tok / a.L;
        const int l = static_cast<int>(tok - n * a.L);
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const int H = side ? a.Hk : a.Hq, h0 = max(lo - (side ? a.Hq : 0), 0), heads = min(lo + sh.heads - (side ? a.Hq : 0), H) - h0;
            if (heads > 0) {
                const long long batch = side ? a.k_batch : a.q_batch, row = side ? a.k_row : a.q_row;
                const T* src = static_cast<const T*>(side ? a.k : a.q) + n * batch + l * row + static_cast<long long>(h0) * a.D;
                const int items = count * heads;
                Walk at_head(heads, wp.grp, wp.hpw);
                uint4 raw[2];
                auto fetch = [&](int it) {
                    const bool on = it < items;
                    load_pieces<T>(raw, src + (on ? ahead(a.L, l, at_head.t, batch, row) + at_head.h * a.D : 0), wp.at, on ? wp.nchunk : 0);
                };
                fetch(wp.grp);
                Lane<T> w;
                uint4 raw_w[2];
                load_weight<T>(raw_w, side ? a.wk : a.wq, wp.at, wp.nchunk);
                w.from(raw_w);
                if (side == 0 || lo >= a.Hq) wp.angles(a, tok, count);
                T* out = (side ? ko : qo) + (tok * H + h0) * a.D;
                for (int at = 0; at < items; at += wp.hpw) {  // whole warps: the lanes shuffle
                    Lane<T> x;
                    x.from(raw);
                    // (a unit's tokens are few; a group past the last item turns zeros)
                    const int tx = min(at_head.t, count - 1), to = (at_head.t * H + at_head.h) * a.D;
                    at_head.next();
                    if (at + wp.hpw < items) fetch(at + wp.hpw + wp.grp);
                    F2 ss = 0;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) ss = fma2(x.f[c][e], x.f[c][e], ss);
                    const float2 sq = unf2(ss);
                    const float s = rsqrtf(fmaf(group_sum(sq.x + sq.y, sh.lph), inv_d, a.eps));
                    const F2 s2 = f2(s, s);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) x.f[c][e] = mul2(mul2(x.f[c][e], s2), w.f[c][e]);
                    wp.turn(x, a, tx, 1.f);
                    if (at + wp.grp < items) x.store(out + to, wp.at, wp.nchunk);
                }
            }
        }
    }
}

// gx, and this CTA's sums of gw: part[cta][2][D] (queries, keys).
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, kBackwardCtas)
    qknorm_backward_kernel(QkNormArgs a, Shape sh, const T* __restrict__ gqo, const T* __restrict__ gko,
                           T* __restrict__ gq, T* __restrict__ gk, double* __restrict__ part) {
    constexpr int E = Elem<T>::per16;
    extern __shared__ __align__(16) float qk_smem[];
    Warp<T, MODE> wp(a, sh, qk_smem);
    const long long total = static_cast<long long>(a.N) * a.L;
    const float inv_d = 1.f / a.D;
    F2 acc[2][2][E / 2] = {};  // queries' and keys' sums of the lane's entries
    const Units un(sh, total);
    for (long long u = un.at; u < un.end; u += un.step) {
        const bool run = sh.chunks == 1;
        const long long tok = run ? u : u / sh.chunks;
        const int count = run ? static_cast<int>(un.end - u < sh.tokens ? un.end - u : sh.tokens) : 1;
        const int lo = run ? 0 : static_cast<int>(u % sh.chunks) * sh.heads;
        const long long n = tok / a.L;
        const int l = static_cast<int>(tok - n * a.L);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int H = side ? a.Hk : a.Hq, h0 = max(lo - (side ? a.Hq : 0), 0), heads = min(lo + sh.heads - (side ? a.Hq : 0), H) - h0;
            if (heads > 0) {
                const T* up = (side ? gko : gqo) + (tok * H + h0) * a.D;
                const long long batch = side ? a.k_batch : a.q_batch, row = side ? a.k_row : a.q_row;
                const T* src = static_cast<const T*>(side ? a.k : a.q) + n * batch + l * row + static_cast<long long>(h0) * a.D;
                const int items = count * heads;
                Walk at_head(heads, wp.grp, wp.hpw);
                uint4 raw_x[2], raw_g[2];
                auto fetch = [&](int it) {
                    const bool on = it < items;
                    load_pieces<T>(raw_x, src + (on ? ahead(a.L, l, at_head.t, batch, row) + at_head.h * a.D : 0), wp.at, on ? wp.nchunk : 0);
                    load_pieces<T>(raw_g, up + (on ? (at_head.t * H + at_head.h) * a.D : 0), wp.at, on ? wp.nchunk : 0);
                };
                fetch(wp.grp);
                uint4 raw_w[2];
                load_weight<T>(raw_w, side ? a.wk : a.wq, wp.at, wp.nchunk);
                if (side == 0 || lo >= a.Hq) wp.angles(a, tok, count);
                for (int at = 0; at < items; at += wp.hpw) {
                    Lane<T> x, g;
                    x.from(raw_x);
                    g.from(raw_g);
                    // (a unit's tokens are few; a group past the last item turns zeros)
                    const int tx = min(at_head.t, count - 1), to = (at_head.t * H + at_head.h) * a.D;
                    at_head.next();
                    if (at + wp.hpw < items) fetch(at + wp.hpw + wp.grp);
                    wp.turn(g, a, tx, -1.f);
                    Lane<T> w;
                    w.from(raw_w);
                    F2 ss = 0, gx = 0;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) {
                            ss = fma2(x.f[c][e], x.f[c][e], ss);
                            gx = fma2(mul2(g.f[c][e], w.f[c][e]), x.f[c][e], gx);
                        }
                    const float2 sq = unf2(ss), sg = unf2(gx);
                    const float s = rsqrtf(fmaf(group_sum(sq.x + sq.y, sh.lph), inv_d, a.eps));
                    const float back = s * (s * (group_sum(sg.x + sg.y, sh.lph) * inv_d));  // (s^2 may pass the largest number)
                    const F2 s2 = f2(s, s), back2 = f2(-back, -back);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) {  // (a head past the last has x = g = 0)
                            acc[side][c][e] = fma2(g.f[c][e], mul2(x.f[c][e], s2), acc[side][c][e]);
                            x.f[c][e] = mul2(s2, fma2(x.f[c][e], back2, mul2(g.f[c][e], w.f[c][e])));
                        }
                    if (at + wp.grp < items) x.store((side ? gk : gq) + (tok * H + h0) * a.D + to, wp.at, wp.nchunk);
                }
            }
        }
    }
    // the CTA's sums: lane groups and warps in a fixed order, in 64 bits, as the sum of the CTAs' (in 32 bits an fp32
    // gradient was off by 2.1 times what its rounding alone leaves; what a lane adds up stays in 32)
    if (!part) return;
    float* bufs = qk_smem + kWarps * kMaxPairs * 2;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (wp.at[c] < wp.nchunk)
#pragma unroll
                for (int e = 0; e < E / 2; ++e) *reinterpret_cast<float2*>(wp.buf + wp.at[c] * E + 2 * e) = unf2(acc[side][c][e]);
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += kThreads) {
            double s = 0.0;
            for (int w = 0; w < kWarps * wp.hpw; ++w) s += bufs[w * a.D + d];
            part[(static_cast<long long>(blockIdx.x) * 2 + side) * a.D + d] = s;
        }
    }
}

// gw[d] = the sum of the CTAs' parts: a warp per entry.
template <typename T>
__global__ void __launch_bounds__(kThreads) qknorm_weights_kernel(const double* __restrict__ part, int ctas, int D,
                                                                  T* __restrict__ gwq, T* __restrict__ gwk) {
    const int e = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= 2 * D) return;
    double s = 0.0;
    for (int c = lane; c < ctas; c += 32 * 16) {  // sixteen loads at a time: one batch mostly
        double v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = c + 32 * u < ctas ? __ldg(part + static_cast<long long>(c + 32 * u) * 2 * D + e) : 0.0;
#pragma unroll
        for (int u = 0; u < 16; ++u) s += v[u];
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    T* to = e < D ? gwq : gwk;
    if (lane == 0 && to) to[e < D ? e : e - D] = from_f32<T>(static_cast<float>(s));
}

Shape shape_of(const QkNormArgs& a, int elems, int ctas) {
    Shape s;
    const int nchunk = a.D / elems, H = a.Hq + a.Hk;
    s.mode = !a.R ? kNone : a.interleaved ? kNeighbours : (a.R / 2) % elems ? kExchange : kHalves;
    s.apart = s.mode == kHalves ? a.R / 2 / elems : 0;
    // lanes: one for each pair of matching pieces, one for each two of the rest
    const int lanes = s.apart + (nchunk - 2 * s.apart + 1) / 2;
    s.lph = 1;
    while (s.lph < lanes) s.lph *= 2;
    const int hpw = 32 / s.lph;
    const long long total = static_cast<long long>(a.N) * a.L, busy = static_cast<long long>(ctas) * kWarps * kBandSms;  // all warps there is room for
    // some sixteen steps of a warp for the angles of as many tokens; where tokens are too few for the
    // warps, a token's heads are split
    s.tokens = static_cast<int>(std::max<long long>(1, std::min<long long>(16LL * hpw / H, (total + busy - 1) / busy)));
    if (a.R) s.tokens = std::min(s.tokens, kMaxPairs / (a.R / 2));
    const int groups = (H + hpw - 1) / hpw;
    s.chunks = total >= busy ? 1 : static_cast<int>(std::min<long long>(groups, (busy + total - 1) / std::max<long long>(total, 1)));
    s.heads = s.chunks == 1 ? H : (groups + s.chunks - 1) / s.chunks * hpw;
    s.chunks = (H + s.heads - 1) / s.heads;
    s.units = total * s.chunks;
    s.grid = static_cast<int>(std::min<long long>((s.units + kWarps - 1) / kWarps, static_cast<long long>(ctas) * kBandSms));
    return s;
}

size_t smem_bytes(const QkNormArgs& a, const Shape& s) {
    return (static_cast<size_t>(kWarps) * kMaxPairs * 2 + static_cast<size_t>(kWarps) * (32 / s.lph) * a.D) * sizeof(float);
}

template <typename T>
cudaError_t forward_typed(const QkNormArgs& a, void* qo, void* ko, cudaStream_t stream) {
    const Shape s = shape_of(a, Elem<T>::per16, kForwardCtas);
    const auto kernel = s.mode == kNone ? qknorm_forward_kernel<T, kNone> : s.mode == kHalves ? qknorm_forward_kernel<T, kHalves>
                        : s.mode == kNeighbours ? qknorm_forward_kernel<T, kNeighbours> : qknorm_forward_kernel<T, kExchange>;
    kernel<<<s.grid, kThreads, smem_bytes(a, s), stream>>>(a, s, static_cast<T*>(qo), static_cast<T*>(ko));
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(const QkNormArgs& a, const void* gqo, const void* gko, void* gq, void* gk, void* gwq,
                           void* gwk, void* ws, cudaStream_t stream) {
    const Shape s = shape_of(a, Elem<T>::per16, kBackwardCtas);
    double* part = (gwq || gwk) ? static_cast<double*>(ws) : nullptr;
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
    const Shape s = shape_of(a, a.dtype == 0 ? 4 : 8, kBackwardCtas);
    return (static_cast<size_t>(s.grid) * 2 * a.D * sizeof(double) + 255) / 256 * 256;
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
