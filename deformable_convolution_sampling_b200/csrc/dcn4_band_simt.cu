// dcn4_band_simt.cu — the band attention in fp32, on the fp32 pipes.
//
// Forward, one pass over the visible keys with a running maximum m and sum l:
//     s = scale q.k + b,  m' = max(m, s),  l = l e^(m-m') + e^(s-m'),  o likewise;  out = o / l,
//     lse = m + log l.
// Backward, recomputing p = e^(s - lse):
//     D = g.out,  ds = p (g.v - D),  gq = scale ds k,  gk = scale ds^T q,  gv = p^T g,
//     gbias[b] = the sum of ds over the pairs of bucket b.
// A CTA owns 64 rows (a row is a query of one of the G heads that share a key
// head, so each tile of keys serves them all) or 64 keys, and walks the 64-wide
// tiles of the other side that its band touches; every product is a 4 x 4 (or
// 4 x 8) tile of registers a thread fed by float4 reads of shared memory: 64
// FMAs to 8 reads.  Bound by latency at a few tiles a CTA (2 x 333 rows of 40, window 121, with
// a bias: forward 19 us, gq 26, gk and gv 29), by the fp32 pipe and shared memory beyond (4 x
// 500 x 500, 8 heads of 128: 156 us, 26 TFLOP/s).  No atomics: gk and gv are summed
// by the CTAs of their keys, gq by the CTAs of its rows, where those are few in ranges
// of the other side that a second kernel adds up, gbias along diagonals and then by
// buckets, all in a fixed order.
#include <algorithm>

#include "dcn4_band_parts.cuh"
#include "dcn4_common.cuh"

namespace dcn4 {
namespace {

constexpr int kB = 64;        // rows and keys of a tile
constexpr int kThreads = 256;
constexpr int kPL = kB + 4;   // row length of the probability tile

// 64 rows of D (padded to DP) elements into shared memory as fp32; row(i) gives a
// row's address, or NULL for a row of zeros.
template <typename T, int DP, typename Row>
__device__ __forceinline__ void load_tile(float* dst, int D, Row row) {
    constexpr int E = Elem<T>::per16, C = DP / E, N = kB * C / kThreads;
    uint4 v[N];  // all loads before the first store: one latency a tile
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = threadIdx.x + n * kThreads, r = i / C, c = i - r * C;
        const T* src = row(r);
        v[n] = src && c * E < D ? __ldg(reinterpret_cast<const uint4*>(src + c * E)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = threadIdx.x + n * kThreads, r = i / C, c = i - r * C;
        float2 f[E / 2];
        unpack(v[n], f, T());
        float* d = dst + r * (DP + 4) + c * E;
#pragma unroll
        for (int e = 0; e < E / 4; ++e)
            *reinterpret_cast<float4*>(d + 4 * e) = make_float4(f[2 * e].x, f[2 * e].y, f[2 * e + 1].x, f[2 * e + 1].y);
    }
}

// x[r][c] = sum_{d < D} A[4 ty + r][d] B[tx + 16 c][d]
template <int DP>
__device__ __forceinline__ void product(float (&x)[4][4], const float* A, const float* B, int D, int ty, int tx) {
    constexpr int LD = DP + 4;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[r][c] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 u[4], w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) u[r] = *reinterpret_cast<const float4*>(A + (4 * ty + r) * LD + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * LD + d);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[r][c] = fmaf(u[r].x, w[c].x, x[r][c]);
                x[r][c] = fmaf(u[r].y, w[c].y, x[r][c]);
                x[r][c] = fmaf(u[r].z, w[c].z, x[r][c]);
                x[r][c] = fmaf(u[r].w, w[c].w, x[r][c]);
            }
    }
}

// o[r][4 c + e] += sum_j P[4 ty + r][j] V[j][64 c + 4 tx + e]
template <int DP>
__device__ __forceinline__ void accumulate_rows(float (&o)[4][DP / 16], const float* P, const float* V, int ty, int tx) {
    constexpr int LD = DP + 4;
#pragma unroll 2
    for (int j = 0; j < kB; j += 4) {
        float4 p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4*>(P + (4 * ty + r) * kPL + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(V + (j + jj) * LD + 64 * c + 4 * tx);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float w = jj == 0 ? p[r].x : jj == 1 ? p[r].y : jj == 2 ? p[r].z : p[r].w;
                    o[r][4 * c] = fmaf(w, v.x, o[r][4 * c]);
                    o[r][4 * c + 1] = fmaf(w, v.y, o[r][4 * c + 1]);
                    o[r][4 * c + 2] = fmaf(w, v.z, o[r][4 * c + 2]);
                    o[r][4 * c + 3] = fmaf(w, v.w, o[r][4 * c + 3]);
                }
            }
    }
}

// o[k][4 c + e] += sum_r P[r][4 ty + k] V[r][64 c + 4 tx + e]
template <int DP>
__device__ __forceinline__ void accumulate_keys(float (&o)[4][DP / 16], const float* P, const float* V, int ty, int tx) {
    constexpr int LD = DP + 4;
#pragma unroll 4
    for (int r = 0; r < kB; ++r) {
        const float4 p = *reinterpret_cast<const float4*>(P + r * kPL + 4 * ty);
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(V + r * LD + 64 * c + 4 * tx);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float w = k == 0 ? p.x : k == 1 ? p.y : k == 2 ? p.z : p.w;
                o[k][4 * c] = fmaf(w, v.x, o[k][4 * c]);
                o[k][4 * c + 1] = fmaf(w, v.y, o[k][4 * c + 1]);
                o[k][4 * c + 2] = fmaf(w, v.z, o[k][4 * c + 2]);
                o[k][4 * c + 3] = fmaf(w, v.w, o[k][4 * c + 3]);
            }
        }
    }
}

template <typename T, int DP>
__device__ __forceinline__ void store_rows(T* row, int D, const float (&o)[4][DP / 16], int r, int tx, float f) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = 64 * c + 4 * tx + e;
            if (d < D) row[d] = from_f32<T>(o[r][4 * c + e] * f);
        }
}

__device__ __forceinline__ int bucket_of(const BandArgs& a, int rel) {
    return __ldg(a.buckets + max(-a.M, min(rel, a.M)) + a.M);
}
template <typename T>
__device__ __forceinline__ float bias_of(const BandArgs& a, int rel, int h) {
    const int b = bucket_of(a, rel);
    return static_cast<unsigned>(b) < static_cast<unsigned>(a.nb) ? to_f32(static_cast<const T*>(a.bias)[static_cast<long long>(b) * a.Hq + h]) : 0.f;
}
// The bias of a group's heads by relative position, in shared memory where that fits
// (two loads that wait for one another are a pair's whole arithmetic otherwise).
constexpr int kTableBytes = 24 << 10;
inline int simt_table(const BandArgs& a) {  // floats, 0: none
    const long long n = static_cast<long long>(a.G) * (2 * a.M + 1);
    return a.nb && n * 4 <= kTableBytes ? static_cast<int>(n) : 0;
}
template <typename T>
struct Bias {
    const float* table;  // [G][2 M + 1], or NULL
    __device__ __forceinline__ Bias(const BandArgs& a, float* smem, int floats, int h0) : table(floats ? smem : nullptr) {
        for (int e = threadIdx.x; e < floats; e += kThreads) {
            const int g = e / (2 * a.M + 1);
            smem[e] = bias_of<T>(a, e - g * (2 * a.M + 1) - a.M, h0 + g);
        }
    }
    __device__ __forceinline__ float at(const BandArgs& a, int rel, int g, int h0) const {
        if (!a.nb) return 0.f;
        return table ? table[g * (2 * a.M + 1) + max(-a.M, min(rel, a.M)) + a.M] : bias_of<T>(a, rel, h0 + g);
    }
};

// Maximum and sum over the 16 lanes that share a row.
__device__ __forceinline__ float row_max(float v) {
    for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 2)
    simt_forward_kernel(BandArgs a, int blocks, int splits, int floats, T* __restrict__ out, float* __restrict__ lse, BandPart part) {
    constexpr int LD = DP + 4;
    extern __shared__ __align__(16) float smem[];
    float *Qs = smem, *Ks = Qs + kB * LD, *Vs = Ks + kB * LD, *Ps = Ks;  // P takes the place of K, which its product has read: two CTAs an SM
    const int sp = blockIdx.x % splits, blk = blockIdx.x / splits % blocks, nh = blockIdx.x / splits / blocks;
    const int n = nh / a.Hk, hk = nh - n * a.Hk;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int klen = band_klen(a, n), qlen = band_qlen(a, n), start = band_start(a, n);
    const Bias<T> bias(a, Vs + kB * LD, floats, hk * a.G);
    const int rows = a.Lq * a.G, r0 = blk * kB;
    const int i0 = r0 / a.G, i1 = min((min(r0 + kB, rows) - 1) / a.G, qlen - 1);
    const T* q = static_cast<const T*>(a.q) + n * a.q_batch + static_cast<long long>(hk) * a.G * a.D;
    const T* k = static_cast<const T*>(a.k) + n * a.k_batch + static_cast<long long>(hk) * a.D;
    const T* v = static_cast<const T*>(a.v) + n * a.v_batch + static_cast<long long>(hk) * a.D;
    load_tile<T, DP>(Qs, a.D, [&](int r) -> const T* {
        const int i = (r0 + r) / a.G;
        return r0 + r < rows && i < qlen ? q + i * a.q_row + static_cast<long long>((r0 + r) % a.G) * a.D : nullptr;
    });
    int pos[4], head[4];
    bool live[4];
    float m[4], l[4], o[4][DP / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = r0 + 4 * ty + r;
        live[r] = row < rows && row / a.G < qlen;
        pos[r] = start + row / a.G;
        head[r] = hk * a.G + row % a.G;
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) o[r][c] = 0.f;
    }
    if (i0 <= i1) {
        const BandTiles bt = band_tiles(a, start + i0, start + i1, klen, kB);
        const int cnt = bt.count(), t0 = static_cast<int>(static_cast<long long>(cnt) * sp / splits),
                  t1 = static_cast<int>(static_cast<long long>(cnt) * (sp + 1) / splits);
        for (int t = t0; t < t1; ++t) {
            const int j0 = bt.tile(t) * kB;
            __syncthreads();
            load_tile<T, DP>(Ks, a.D, [&](int j) -> const T* { return j0 + j < klen ? k + (j0 + j) * a.k_row : nullptr; });
            load_tile<T, DP>(Vs, a.D, [&](int j) -> const T* { return j0 + j < klen ? v + (j0 + j) * a.v_row : nullptr; });
            __syncthreads();
            float x[4][4];
            product<DP>(x, Qs, Ks, a.D, ty, tx);
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = j0 + tx + 16 * c;
                    const bool see = live[r] && band_sees(a, pos[r], j, klen);
                    x[r][c] = see ? x[r][c] * a.scale + bias.at(a, j - pos[r], head[r] - hk * a.G, hk * a.G) : -INFINITY;
                    top = fmaxf(top, x[r][c]);
                }
                const float mn = fmaxf(m[r], row_max(top));
                const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every term below is e^-inf = 0
                const float f = expf(m[r] - ref);
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float p = expf(x[r][c] - ref);
                    sum += p;
                    Ps[(4 * ty + r) * kPL + tx + 16 * c] = p;
                }
                l[r] = l[r] * f + row_sum(sum);
                m[r] = mn;
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) o[r][c] *= f;
            }
            __syncthreads();
            accumulate_rows<DP>(o, Ps, Vs, ty, tx);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = r0 + 4 * ty + r;
        if (row >= rows) continue;
        const int i = row / a.G;
        const long long at = (static_cast<long long>(n) * a.Hq + head[r]) * a.Lq + i;
        if (splits > 1) {
            if (tx == 0) part.ml[at * splits + sp] = make_float2(m[r], l[r]);
            store_rows<float, DP>(part.o + (at * splits + sp) * a.D, a.D, o, r, tx, 1.f);
        } else {
            if (tx == 0) lse[at] = l[r] == 0.f ? -INFINITY : m[r] + logf(l[r]);
            T* to = out + ((static_cast<long long>(n) * a.Lq + i) * a.Hq + head[r]) * a.D;
            store_rows<T, DP>(to, a.D, o, r, tx, l[r] == 0.f ? 0.f : 1.f / l[r]);
        }
    }
}

// gq of 64 rows over a range of their keys, their D (into delta), what a probability is formed
// from (refs: e^(s - x) y; lse and 1, or a far row's maximum and the inverse of its sum) and, with a
// bias whose gradient is wanted, the sums of ds along diagonals: diag[CTA][G][2 M + 1], of relative position -M .. M (the ends:
// and beyond).
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads)
    simt_grad_q_kernel(BandArgs a, int blocks, int splits, int floats, const T* __restrict__ out, const float* __restrict__ lse,
                       const T* __restrict__ gout, T* __restrict__ gq, float* __restrict__ delta, float2* __restrict__ refs,
                       float* __restrict__ part, float* __restrict__ diag) {
    constexpr int LD = DP + 4;
    extern __shared__ __align__(16) float smem[];
    float *Qs = smem, *Gs = Qs + kB * LD, *Ks = Gs + kB * LD, *Vs = Ks + kB * LD, *Ps = Vs + kB * LD, *sums = Ps + kB * kPL;
    const int sp = blockIdx.x % splits, blk = blockIdx.x / splits % blocks, nh = blockIdx.x / splits / blocks;
    const int n = nh / a.Hk, hk = nh - n * a.Hk;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int spread = (kB + a.G - 1) / a.G + 1 + kB;  // relative positions of one tile and head at most
    const Bias<T> bias(a, sums + (a.nb ? spread * a.G : 0), floats, hk * a.G);
    const int klen = band_klen(a, n), qlen = band_qlen(a, n), start = band_start(a, n);
    const int rows = a.Lq * a.G, r0 = blk * kB;
    const int i0 = r0 / a.G, ilast = (min(r0 + kB, rows) - 1) / a.G, i1 = min(ilast, qlen - 1);
    const T* q = static_cast<const T*>(a.q) + n * a.q_batch + static_cast<long long>(hk) * a.G * a.D;
    const T* k = static_cast<const T*>(a.k) + n * a.k_batch + static_cast<long long>(hk) * a.D;
    const T* v = static_cast<const T*>(a.v) + n * a.v_batch + static_cast<long long>(hk) * a.D;
    auto dense = [&](int row) { return ((static_cast<long long>(n) * a.Lq + row / a.G) * a.Hq + hk * a.G + row % a.G) * a.D; };
    auto alive = [&](int row) { return row < rows && row / a.G < qlen; };
    load_tile<T, DP>(Qs, a.D, [&](int r) -> const T* {
        return alive(r0 + r) ? q + (r0 + r) / a.G * a.q_row + static_cast<long long>((r0 + r) % a.G) * a.D : nullptr;
    });
    load_tile<T, DP>(Gs, a.D, [&](int r) -> const T* { return alive(r0 + r) ? gout + dense(r0 + r) : nullptr; });
    load_tile<T, DP>(Ks, a.D, [&](int r) -> const T* { return alive(r0 + r) ? out + dense(r0 + r) : nullptr; });
    __syncthreads();
    int pos[4], head[4];
    bool live[4];
    float le[4], weight[4], de[4], o[4][DP / 16];
    bool far = false;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = r0 + 4 * ty + r;
        live[r] = alive(row);
        pos[r] = start + row / a.G;
        head[r] = hk * a.G + row % a.G;
        const long long at = (static_cast<long long>(n) * a.Hq + head[r]) * a.Lq + row / a.G;
        le[r] = live[r] ? band_lse_ref(lse[at]) : 0.f;
        weight[r] = 1.f;
        far |= band_far(le[r]);
        float d = 0.f;
        for (int e = tx; e < DP; e += 16) d = fmaf(Gs[(4 * ty + r) * LD + e], Ks[(4 * ty + r) * LD + e], d);
        de[r] = row_sum(d);
        if (tx == 0 && row < rows && sp == 0) delta[at] = de[r];
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) o[r][c] = 0.f;
    }
    float* mine = diag + static_cast<long long>(blockIdx.x) * a.G * (2 * a.M + 1);
    if (diag)
        for (int e = threadIdx.x; e < a.G * (2 * a.M + 1); e += kThreads) mine[e] = 0.f;
    far = __syncthreads_or(far);
    if (i0 <= i1) {
        const BandTiles bt = band_tiles(a, start + i0, start + i1, klen, kB);
        if (far) {  // the rows' maxima and sums over all of their keys, in every CTA of a split row
            float l[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) le[r] = -INFINITY, l[r] = 0.f;
            for (int t = 0; t < bt.count(); ++t) {
                const int j0 = bt.tile(t) * kB;
                __syncthreads();
                load_tile<T, DP>(Ks, a.D, [&](int j) -> const T* { return j0 + j < klen ? k + (j0 + j) * a.k_row : nullptr; });
                __syncthreads();
                float x[4][4];
                product<DP>(x, Qs, Ks, a.D, ty, tx);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int j = j0 + tx + 16 * c;
                        const bool see = live[r] && band_sees(a, pos[r], j, klen);
                        x[r][c] = see ? x[r][c] * a.scale + bias.at(a, j - pos[r], head[r] - hk * a.G, hk * a.G) : -INFINITY;
                        top = fmaxf(top, x[r][c]);
                    }
                    const float to = fmaxf(le[r], row_max(top)), ref = to == -INFINITY ? 0.f : to;
                    float sum = 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum += expf(x[r][c] - ref);
                    l[r] = l[r] * expf(le[r] - ref) + row_sum(sum);
                    le[r] = to;
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                le[r] = l[r] != 0.f ? le[r] : INFINITY;
                weight[r] = l[r] != 0.f ? 1.f / l[r] : 1.f;
            }
        }
        const int cnt = bt.count(), t0 = static_cast<int>(static_cast<long long>(cnt) * sp / splits),
                  t1 = static_cast<int>(static_cast<long long>(cnt) * (sp + 1) / splits);
        for (int t = t0; t < t1; ++t) {
            const int j0 = bt.tile(t) * kB;
            __syncthreads();
            load_tile<T, DP>(Ks, a.D, [&](int j) -> const T* { return j0 + j < klen ? k + (j0 + j) * a.k_row : nullptr; });
            load_tile<T, DP>(Vs, a.D, [&](int j) -> const T* { return j0 + j < klen ? v + (j0 + j) * a.v_row : nullptr; });
            __syncthreads();
            float x[4][4], y[4][4];
            product<DP>(x, Qs, Ks, a.D, ty, tx);
            product<DP>(y, Gs, Vs, a.D, ty, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = j0 + tx + 16 * c;
                    float ds = 0.f;
                    if (live[r] && band_sees(a, pos[r], j, klen)) {
                        const float s = x[r][c] * a.scale + bias.at(a, j - pos[r], head[r] - hk * a.G, hk * a.G);
                        ds = expf(s - le[r]) * weight[r] * (y[r][c] - de[r]);
                    }
                    Ps[(4 * ty + r) * kPL + tx + 16 * c] = ds;
                }
            __syncthreads();
            accumulate_rows<DP>(o, Ps, Ks, ty, tx);
            if (diag) {
                // the tile's sums along each head's diagonals (all pairs of one relative position): one thread
                // adds a diagonal's to its place, one warp those of a head beyond M
                const int nd = ilast - i0 + kB;  // relative positions j0 - (start + ilast) ...
                const int rel0 = j0 - start - ilast;
                for (int e = threadIdx.x; e < nd * a.G; e += kThreads) {
                    const int g = e / nd, d = e - g * nd, rel = rel0 + d;
                    float s = 0.f;
                    for (int i = i0; i <= ilast; ++i) {
                        const int j = d + i - ilast, row = i * a.G + g - r0;
                        if (j >= 0 && j < kB && row >= 0 && row < kB) s += Ps[row * kPL + j];
                    }
                    sums[e] = s;
                    if (rel > -a.M && rel < a.M) mine[g * (2 * a.M + 1) + rel + a.M] += s;
                }
                if (rel0 > -a.M && rel0 + nd - 1 < a.M) continue;
                __syncthreads();
                for (int e = threadIdx.x >> 5; e < 2 * a.G; e += kThreads / 32) {
                    const int g = e >> 1, lane = threadIdx.x & 31;
                    float s = 0.f;
                    for (int d = lane; d < nd; d += 32)
                        if (e & 1 ? rel0 + d >= a.M : rel0 + d <= -a.M) s += sums[g * nd + d];
                    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    if (lane == 0) mine[g * (2 * a.M + 1) + (e & 1 ? 2 * a.M : 0)] += s;
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = r0 + 4 * ty + r;
        if (row >= rows) continue;
        if (tx == 0 && sp == 0) refs[(static_cast<long long>(n) * a.Hq + head[r]) * a.Lq + row / a.G] = make_float2(le[r], weight[r]);
        if (splits > 1)
            store_rows<float, DP>(part + sp * band_rows(a) * a.D + dense(row), a.D, o, r, tx, a.scale);
        else
            store_rows<T, DP>(gq + dense(row), a.D, o, r, tx, a.scale);
    }
}

// gk and gv of 64 keys over a range of the queries that see them.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads)
    simt_grad_kv_kernel(BandArgs a, int blocks, int splits, int floats, const float2* __restrict__ refs, const T* __restrict__ gout,
                        const float* __restrict__ delta, T* __restrict__ gk, T* __restrict__ gv, float* __restrict__ part) {
    constexpr int LD = DP + 4;
    extern __shared__ __align__(16) float smem[];
    float *Qs = smem, *Gs = Qs + kB * LD, *Ks = Gs + kB * LD, *Vs = Ks + kB * LD, *Ps = Vs + kB * LD, *Ds = Ps + kB * kPL;
    const int sp = blockIdx.x % splits, blk = blockIdx.x / splits % blocks, nh = blockIdx.x / splits / blocks;
    const int n = nh / a.Hk, hk = nh - n * a.Hk;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const Bias<T> bias(a, Ds + kB * kPL, floats, hk * a.G);
    const int klen = band_klen(a, n), qlen = band_qlen(a, n), start = band_start(a, n);
    const int j0 = blk * kB;
    const T* q = static_cast<const T*>(a.q) + n * a.q_batch + static_cast<long long>(hk) * a.G * a.D;
    const T* k = static_cast<const T*>(a.k) + n * a.k_batch + static_cast<long long>(hk) * a.D;
    const T* v = static_cast<const T*>(a.v) + n * a.v_batch + static_cast<long long>(hk) * a.D;
    load_tile<T, DP>(Ks, a.D, [&](int j) -> const T* { return j0 + j < klen ? k + (j0 + j) * a.k_row : nullptr; });
    load_tile<T, DP>(Vs, a.D, [&](int j) -> const T* { return j0 + j < klen ? v + (j0 + j) * a.v_row : nullptr; });
    float ok[4][DP / 16], ov[4][DP / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) ok[r][c] = ov[r][c] = 0.f;
    int ilo = 0, ihi = 0;
    if (j0 < klen) band_queries(a, start, qlen, j0, min(j0 + kB, klen), ilo, ihi);
    const int first = ilo * a.G, last = ihi * a.G, tiles = (last - first + kB - 1) / kB;
    const int rlo = first + static_cast<int>(static_cast<long long>(tiles) * sp / splits) * kB,
              rhi = min(last, first + static_cast<int>(static_cast<long long>(tiles) * (sp + 1) / splits) * kB);
    for (int r0 = rlo; r0 < rhi; r0 += kB) {
        __syncthreads();
        load_tile<T, DP>(Qs, a.D, [&](int r) -> const T* {
            return r0 + r < rhi ? q + (r0 + r) / a.G * a.q_row + static_cast<long long>((r0 + r) % a.G) * a.D : nullptr;
        });
        load_tile<T, DP>(Gs, a.D, [&](int r) -> const T* {
            return r0 + r < rhi ? gout + ((static_cast<long long>(n) * a.Lq + (r0 + r) / a.G) * a.Hq + hk * a.G + (r0 + r) % a.G) * a.D : nullptr;
        });
        __syncthreads();
        float x[4][4], y[4][4];
        product<DP>(x, Qs, Ks, a.D, ty, tx);
        product<DP>(y, Gs, Vs, a.D, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = r0 + 4 * ty + r, i = row / a.G, h = hk * a.G + row % a.G, pos = start + i;
            const bool live = row < rhi;
            const long long at = (static_cast<long long>(n) * a.Hq + h) * a.Lq + i;
            const float2 ref = live ? refs[at] : make_float2(0.f, 1.f);
            const float de = live ? delta[at] : 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = j0 + tx + 16 * c;
                float p = 0.f;
                if (live && band_sees(a, pos, j, klen))
                    p = expf(x[r][c] * a.scale + bias.at(a, j - pos, h - hk * a.G, hk * a.G) - ref.x) * ref.y;
                Ps[(4 * ty + r) * kPL + tx + 16 * c] = p;
                Ds[(4 * ty + r) * kPL + tx + 16 * c] = p == 0.f ? 0.f : p * (y[r][c] - de);
            }
        }
        __syncthreads();
        accumulate_keys<DP>(ov, Ps, Gs, ty, tx);
        accumulate_keys<DP>(ok, Ds, Qs, ty, tx);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int j = j0 + 4 * ty + r;
        if (j >= a.Lk) continue;
        const long long at = ((static_cast<long long>(n) * a.Lk + j) * a.Hk + hk) * a.D;
        if (splits > 1) {
            const long long all = static_cast<long long>(a.N) * a.Lk * a.Hk * a.D;
            store_rows<float, DP>(part + 2 * sp * all + at, a.D, ok, r, tx, a.scale);
            store_rows<float, DP>(part + (2 * sp + 1) * all + at, a.D, ov, r, tx, 1.f);
        } else {
            store_rows<T, DP>(gk + at, a.D, ok, r, tx, a.scale);
            store_rows<T, DP>(gv + at, a.D, ov, r, tx, 1.f);
        }
    }
}

// out[e] = the sum of its parts, `apart` elements from one another, in order.
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int parts, long long apart, long long n, T* __restrict__ out) {
    const long long e = 4 * (blockIdx.x * 256ll + threadIdx.x);
    if (e >= n) return;  // n is a multiple of 4
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(part + p * apart + e));
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    out[e] = from_f32<T>(s.x);
    out[e + 1] = from_f32<T>(s.y);
    out[e + 2] = from_f32<T>(s.z);
    out[e + 3] = from_f32<T>(s.w);
}

template <int DP>
constexpr size_t tiles_smem(int tiles, int probs) {
    return (static_cast<size_t>(tiles) * kB * (DP + 4) + static_cast<size_t>(probs) * kB * kPL) * sizeof(float);
}

// Ranges along the other side for `ctas` CTAs of `tiles` tiles each: up to one CTA an SM,
// down to a tile each (at 333 x 333 keys, grad_kv's 24 CTAs of up to 11 tiles took 164 us,
// 144 of up to 2 take 32).
int split_count(long long ctas, long long tiles) {
    return static_cast<int>(std::max<long long>(1, std::min<long long>(kBandSms / std::max<long long>(ctas, 1), std::min<long long>(tiles, 256))));
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <typename T, int DP>
cudaError_t forward_typed(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    const int blocks = simt_row_blocks(a), splits = simt_splits(a), floats = simt_table(a);
    const size_t smem = tiles_smem<DP>(3, 0) + floats * sizeof(float);
    cudaError_t e = allow_smem(simt_forward_kernel<T, DP>, smem);
    if (e != cudaSuccess) return e;
    const BandPart part = band_part(a, splits, ws);
    simt_forward_kernel<T, DP><<<static_cast<unsigned>(static_cast<long long>(a.N) * a.Hk * blocks * splits), kThreads, smem, stream>>>(
        a, blocks, splits, floats, static_cast<T*>(out), lse, part);
    e = cudaGetLastError();
    if (e != cudaSuccess || splits == 1) return e;
    return launch_band_join(a, splits, part, 1.f, out, lse, stream);
}

// Ranges of the queries that see a key tile (splits of grad_kv).
int kv_splits(const BandArgs& a) {
    const long long ctas = static_cast<long long>(a.N) * a.Hk * ((a.Lk + kB - 1) / kB);
    const long long reach = std::min<long long>(a.Lq, static_cast<long long>(std::min(a.left, kBandMaxLen)) + std::min(a.right, kBandMaxLen) + kB);
    return split_count(ctas, ((a.sinks ? static_cast<long long>(a.Lq) : reach) * a.G + kB - 1) / kB);
}
size_t up256(size_t b) { return (b + 255) / 256 * 256; }
// Workspace of the backward: delta, refs, parts (grad_q's, then grad_kv's in the same place), diagonal sums, their sums by head.
struct Workspace {
    size_t delta, refs, part, diag, sums;
    explicit Workspace(const BandArgs& a) {
        const int sq = simt_splits(a), sk = kv_splits(a);
        const size_t nq = static_cast<size_t>(band_rows(a)) * a.D, nk = static_cast<size_t>(a.N) * a.Lk * a.Hk * a.D;
        delta = up256(static_cast<size_t>(band_rows(a)) * sizeof(float));
        refs = up256(static_cast<size_t>(band_rows(a)) * sizeof(float2));
        part = up256(std::max(sq > 1 ? nq * sq : 0, sk > 1 ? 2 * nk * sk : 0) * sizeof(float));
        const size_t ctas = static_cast<size_t>(a.N) * a.Hk * simt_row_blocks(a) * sq;
        diag = a.nb ? up256(ctas * a.G * (2 * a.M + 1) * sizeof(float)) : 0;
        sums = a.nb ? up256(band_sum_bytes(a)) : 0;
    }
};

template <typename T>
cudaError_t launch_sum_parts(const float* part, int parts, long long apart, long long n, void* out, cudaStream_t stream) {
    sum_parts_kernel<T><<<static_cast<unsigned>((n / 4 + 255) / 256), 256, 0, stream>>>(part, parts, apart, n, static_cast<T*>(out));
    return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t backward_typed(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq, void* gk,
                           void* gv, void* gbias, void* ws, cudaStream_t stream) {
    const Workspace w(a);
    char* at = static_cast<char*>(ws);
    float* delta = reinterpret_cast<float*>(at);
    float2* refs = reinterpret_cast<float2*>(at += w.delta);
    float* part = reinterpret_cast<float*>(at += w.refs);
    float* diag = a.nb && gbias ? reinterpret_cast<float*>(at += w.part) : nullptr;
    float* sums = diag ? reinterpret_cast<float*>(at += w.diag) : nullptr;
    const int blocks = simt_row_blocks(a), sq = simt_splits(a), sk = kv_splits(a), floats = simt_table(a);
    const int spread = (kB + a.G - 1) / a.G + 1 + kB;  // relative positions of one tile and head at most
    const size_t smem_q = tiles_smem<DP>(4, 1) + (a.nb ? (static_cast<size_t>(spread) * a.G + floats) * sizeof(float) : 0),
                 smem_kv = tiles_smem<DP>(4, 2) + floats * sizeof(float);
    cudaError_t e = allow_smem(simt_grad_q_kernel<T, DP>, smem_q);
    if (e == cudaSuccess) e = allow_smem(simt_grad_kv_kernel<T, DP>, smem_kv);
    if (e != cudaSuccess) return e;
    const long long ctas = static_cast<long long>(a.N) * a.Hk * blocks * sq;
    simt_grad_q_kernel<T, DP><<<static_cast<unsigned>(ctas), kThreads, smem_q, stream>>>(
        a, blocks, sq, floats, static_cast<const T*>(out), lse, static_cast<const T*>(gout), static_cast<T*>(gq), delta, refs, part, diag);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long nq = band_rows(a) * a.D, nk = static_cast<long long>(a.N) * a.Lk * a.Hk * a.D;
    if (sq > 1 && (e = launch_sum_parts<T>(part, sq, nq, nq, gq, stream)) != cudaSuccess) return e;
    const int kblocks = (a.Lk + kB - 1) / kB;
    simt_grad_kv_kernel<T, DP><<<static_cast<unsigned>(static_cast<long long>(a.N) * a.Hk * kblocks * sk), kThreads, smem_kv, stream>>>(
        a, kblocks, sk, floats, refs, static_cast<const T*>(gout), delta, static_cast<T*>(gk), static_cast<T*>(gv), part);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (sk > 1) {
        if ((e = launch_sum_parts<T>(part, sk, 2 * nk, nk, gk, stream)) != cudaSuccess) return e;
        if ((e = launch_sum_parts<T>(part + nk, sk, 2 * nk, nk, gv, stream)) != cudaSuccess) return e;
    }
    return diag ? launch_band_bias_sum(a, blocks * sq, 1, diag, sums, gbias, stream) : cudaSuccess;
}

}  // namespace

int simt_row_blocks(const BandArgs& a) {
    return static_cast<int>((static_cast<long long>(a.Lq) * a.G + kB - 1) / kB);
}
int simt_splits(const BandArgs& a) {
    const long long span = std::min<long long>(a.Lk, static_cast<long long>(std::min(a.left, kBandMaxLen)) +
                                                         std::min(a.right, kBandMaxLen) + std::min(a.Lq, kB / a.G + 2) + a.sinks);
    return split_count(static_cast<long long>(a.N) * a.Hk * simt_row_blocks(a), (span + kB - 1) / kB);
}
size_t band_simt_backward_workspace(const BandArgs& a, bool want_bias) {
    const Workspace w(a);
    return w.delta + w.refs + w.part + (want_bias ? w.diag + w.sums : 0);
}

cudaError_t launch_band_simt_forward(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    return a.D > 64 ? forward_typed<float, 128>(a, out, lse, ws, stream) : forward_typed<float, 64>(a, out, lse, ws, stream);
}

cudaError_t launch_band_simt_backward(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq,
                                      void* gk, void* gv, void* gbias, void* ws, cudaStream_t stream) {
    return a.D > 64 ? backward_typed<float, 128>(a, out, lse, gout, gq, gk, gv, gbias, ws, stream)
                    : backward_typed<float, 64>(a, out, lse, gout, gq, gk, gv, gbias, ws, stream);
}

}  // namespace dcn4
