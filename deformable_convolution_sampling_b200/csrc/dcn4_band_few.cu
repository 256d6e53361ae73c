// dcn4_band_few.cu — the band attention's forward for up to 16 rows (queries times
// heads that share a key head) over a long cache, 16-bit types: the serving form.
//
// Bound by reading the keys and values once.  Each warp streams 16 keys at a time
// through a ring of its own in shared memory (cp.async, no barriers) into the registers
// of mma.m16n8k16 (M: the rows, so that one read of a key serves all of them).  A
// product's inner index may be taken in any order, and so may the columns of a result,
// so that every read of shared memory is 16 bytes of a row:
//     S = Q K^T   lane (r, c) holds entries 32 q + 8 c .. + 7 of key r (and r + 8), and of
//                 rows r, r + 8 of Q: four entries a K step;
//     O += P V    lane (r, c) holds entries 64 g + 8 r .. + 7 of the keys 2 c, 2 c + 1,
//                 2 c + 8, 2 c + 9; entry t of each goes to column tile t, so a lane's
//                 results are entries 64 g + 8 (2 c + h) .. + 7 of rows r, r + 8.
// The running maximum moves its reference only when it has outgrown it by 2^8 (as in
// the kernel for many rows); p is rounded to the I/O type for its product, all sums
// and statistics are fp32.  Four warps join in shared memory, CTAs through parts.
// (Loads straight into registers left 6 KB a warp in flight: 3.7 TB/s.  The kernel for
// many rows, which could take these calls too: 4.8 TB/s, this one 5.9, at 16 caches of
// 16384 tokens, 8 key heads of 128; 2 caches of 1000 tokens: 12.1 us, this one 8.7.)
#include <cmath>

#include "dcn4_band_tc.cuh"

namespace dcn4 {
namespace {

using tc::kLog2e;
using tc::pack2;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16 * kWarps;  // keys of a step: 16 a warp
constexpr int kRows = 16;
constexpr float kRescale = 8.f;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint4 piece(const T* p, bool on) {
    return on ? ld_stream(p) : make_uint4(0u, 0u, 0u, 0u);
}

// Where a row's 16-byte pieces lie: permuted so that the eight lanes of a read's phase
// (two rows and four pieces of K, four rows and two pieces of V) meet eight bank groups.
__device__ __forceinline__ int k_place(int row) { return (row & 1) << 2 | ((row >> 1) & 3); }
__device__ __forceinline__ int v_place(int row) { return ((row >> 1) & 3) << 1; }

// KG: groups of 32 entries a head has (2 or 4).
template <int KG>
struct Cfg {
    static constexpr int pieces = 4 * KG, row = pieces * 16;     // of a key: 16-byte pieces, bytes
    static constexpr int stages = KG == 4 ? 3 : 4, stage = 2 * 16 * row;
    static constexpr int ctas = KG == 4 ? 2 : 3;
    static constexpr int smem = kWarps * stages * stage;
};

template <typename T, int KG>
__global__ void __launch_bounds__(kThreads, Cfg<KG>::ctas)
    few_kernel(BandArgs a, int splits, T* __restrict__ out, float* __restrict__ lse, BandPart part) {
    using C = Cfg<KG>;
    constexpr int VG = KG / 2, DP = 32 * KG, S = C::stages;
    extern __shared__ __align__(128) unsigned char few_smem[];
    float (*s_o)[kRows][DP + 4] = reinterpret_cast<float (*)[kRows][DP + 4]>(few_smem);  // after the last step
    static_assert(sizeof(float) * kWarps * kRows * (DP + 4) <= C::smem, "");
    __shared__ float2 s_ml[kWarps][kRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int sp = blockIdx.x % splits, nh = blockIdx.x / splits, n = nh / a.Hk, hk = nh - n * a.Hk;
    const int klen = band_klen(a, n), qlen = band_qlen(a, n), start = band_start(a, n), rows = a.Lq * a.G;
    const T* q = static_cast<const T*>(a.q) + n * a.q_batch + static_cast<long long>(hk) * a.G * a.D;
    const T* k = static_cast<const T*>(a.k) + n * a.k_batch + static_cast<long long>(hk) * a.D;
    const T* v = static_cast<const T*>(a.v) + n * a.v_batch + static_cast<long long>(hk) * a.D;

    uint32_t qf[2 * KG][4];
    int pos[2], head[2];
    bool live[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = r + 8 * h, i = row / a.G;
        head[h] = hk * a.G + row - i * a.G;
        live[h] = row < rows && i < qlen;
        pos[h] = start + i;
        const T* src = q + i * a.q_row + static_cast<long long>(row - i * a.G) * a.D;
#pragma unroll
        for (int g = 0; g < KG; ++g) {
            const uint4 w = piece(src + g * 32 + c * 8, live[h] && g * 32 + c * 8 < a.D);
            qf[2 * g][h] = w.x;
            qf[2 * g][2 + h] = w.y;
            qf[2 * g + 1][h] = w.z;
            qf[2 * g + 1][2 + h] = w.w;
        }
    }
    int t0 = 0, t1 = 0;
    BandTiles bt{0, 0, 0};
    if (qlen > 0) {
        bt = band_tiles(a, start, start + qlen - 1, klen, kTile);
        const long long cnt = bt.count();
        t0 = static_cast<int>(cnt * sp / splits);
        t1 = static_cast<int>(cnt * (sp + 1) / splits);
    }
    // a lane copies one piece of every (32 / pieces)-th of its warp's 16 keys
    const unsigned char* ring = few_smem + warp * S * C::stage;
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    constexpr int each = 32 / C::pieces;
    const int lp = lane % C::pieces, lr = lane / C::pieces;
    const bool in = lp * 8 < a.D;
    auto load = [&](int t) {
        if (t < t1) {
            const int j0 = bt.tile(t) * kTile + warp * 16 + lr;
            const uint32_t at = ring_at + (t - t0) % S * C::stage;
            const T *ks = k + j0 * a.k_row + lp * 8, *vs = v + j0 * a.v_row + lp * 8;
#pragma unroll
            for (int x = 0; x < 16; x += each) {
                const int row = x + lr;
                const bool on = in && j0 + x < klen;
                asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(at + row * C::row + ((lp ^ k_place(row)) << 4)),
                             "l"(on ? ks : k), "r"(on ? 16 : 0) : "memory");
                asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(at + (16 + row) * C::row + ((lp ^ v_place(row)) << 4)),
                             "l"(on ? vs : v), "r"(on ? 16 : 0) : "memory");
                ks += each * a.k_row;
                vs += each * a.v_row;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto bias_at = [&](int rel, int h) {
        const int bk = __ldg(a.buckets + max(-a.M, min(rel, a.M)) + a.M);
        return static_cast<unsigned>(bk) < static_cast<unsigned>(a.nb) ? to_f32(static_cast<const T*>(a.bias)[static_cast<long long>(bk) * a.Hq + head[h]]) : 0.f;
    };
    float behind[2] = {};  // the bias of every key M or more behind
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (a.nb && live[h]) behind[h] = bias_at(-a.M, h);
    float o[VG][8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {};
#pragma unroll
    for (int x = 0; x < S - 1; ++x) load(t0 + x);
    for (int t = t0; t < t1; ++t) {
        const int j0 = bt.tile(t) * kTile + warp * 16;
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();
        load(t + S - 1);  // where the step before this one was
        const unsigned char* at = ring + (t - t0) % S * C::stage;
        float s[2][4] = {};
#pragma unroll
        for (int g = 0; g < KG; ++g)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint4 w = *reinterpret_cast<const uint4*>(at + (8 * x + r) * C::row + (((g * 4 + c) ^ k_place(8 * x + r)) << 4));
                mma<T>(s[x], qf[2 * g], w.x, w.y);
                mma<T>(s[x], qf[2 * g + 1], w.z, w.w);
            }
        float top[2] = {-INFINITY, -INFINITY};
        const bool far = j0 + 15 - start <= -a.M;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int h = e >> 1, j = j0 + 8 * x + 2 * c + (e & 1);
                float w = s[x][e] * a.scale;
                const bool see = live[h] && band_sees(a, pos[h], j, klen);
                if (a.nb && see) w += far ? behind[h] : bias_at(j - pos[h], h);
                s[x][e] = see ? w : -INFINITY;
                top[h] = fmaxf(top[h], s[x][e]);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        }
        if (__any_sync(0xffffffffu, (top[0] - m[0]) * kLog2e > kRescale || (top[1] - m[1]) * kLog2e > kRescale)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float to = fmaxf(m[h], top[h]), f = to == -INFINITY ? 1.f : exp2f((m[h] - to) * kLog2e);
                m[h] = to;
                l[h] *= f;
#pragma unroll
                for (int g = 0; g < VG; ++g)
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        o[g][x][2 * h] *= f;
                        o[g][x][2 * h + 1] *= f;
                    }
            }
        }
        uint32_t p[4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ref = m[h] == -INFINITY ? 0.f : m[h];
                const float lo = exp2f((s[x][2 * h] - ref) * kLog2e), hi = exp2f((s[x][2 * h + 1] - ref) * kLog2e);
                l[h] += lo + hi;
                p[2 * x + h] = pack2<T>(lo, hi);
            }
#pragma unroll
        for (int g = 0; g < VG; ++g) {
            uint32_t w[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = 2 * c + (x & 1) + 8 * (x >> 1);
                const uint4 y = *reinterpret_cast<const uint4*>(at + (16 + row) * C::row + (((g * 8 + r) ^ v_place(row)) << 4));
                w[x][0] = y.x, w[x][1] = y.y, w[x][2] = y.z, w[x][3] = y.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                mma<T>(o[g][2 * x], p, __byte_perm(w[0][x], w[1][x], 0x5410), __byte_perm(w[2][x], w[3][x], 0x5410));
                mma<T>(o[g][2 * x + 1], p, __byte_perm(w[0][x], w[1][x], 0x7632), __byte_perm(w[2][x], w[3][x], 0x7632));
            }
        }
    }
    // join the warps, in the rings' place
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (c == 0) s_ml[warp][r + 8 * h] = make_float2(m[h], l[h]);
#pragma unroll
        for (int g = 0; g < VG; ++g)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float* to = &s_o[warp][r + 8 * h][64 * g + 8 * (2 * c + x)];
                *reinterpret_cast<float4*>(to) = make_float4(o[g][0][2 * h + x], o[g][1][2 * h + x], o[g][2][2 * h + x], o[g][3][2 * h + x]);
                *reinterpret_cast<float4*>(to + 4) = make_float4(o[g][4][2 * h + x], o[g][5][2 * h + x], o[g][6][2 * h + x], o[g][7][2 * h + x]);
            }
    }
    __syncthreads();
    const int pieces = a.D / 4;
    for (int e = tid; e < rows * pieces; e += kThreads) {
        const int row = e / pieces, d = (e - row * pieces) * 4, i = row / a.G;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w][row].x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 ml = s_ml[w][row];
            if (ml.y == 0.f) continue;
            const float f = exp2f((ml.x - ref) * kLog2e);
            const float4 x = *reinterpret_cast<const float4*>(&s_o[w][row][d]);
            ll += ml.y * f;
            s.x = fmaf(x.x, f, s.x), s.y = fmaf(x.y, f, s.y), s.z = fmaf(x.z, f, s.z), s.w = fmaf(x.w, f, s.w);
        }
        const int hq = hk * a.G + row - i * a.G;
        const long long at = (static_cast<long long>(n) * a.Hq + hq) * a.Lq + i;
        if (splits > 1) {
            *reinterpret_cast<float4*>(part.o + (at * splits + sp) * a.D + d) = s;
            if (d == 0) part.ml[at * splits + sp] = make_float2(ll != 0.f ? mm : -INFINITY, ll);
        } else {
            const float inv = ll != 0.f ? 1.f / ll : 0.f;  // (a sum of NaN stays one)
            T* to = out + ((static_cast<long long>(n) * a.Lq + i) * a.Hq + hq) * a.D + d;
            *reinterpret_cast<uint2*>(to) = make_uint2(pack2<T>(s.x * inv, s.y * inv), pack2<T>(s.z * inv, s.w * inv));
            if (d == 0) lse[at] = ll != 0.f ? mm + logf(ll) : -INFINITY;
        }
    }
}

// Enough CTAs for some four rounds (caches of different lengths leave no SM idle for
// long), a step of 64 keys a CTA at least, and no more parts than join quickly.
int few_splits(const BandArgs& a) {
    const long long span = std::min<long long>(band_most_keys(a) + a.Lq, a.Lk), tiles = (span + kTile - 1) / kTile;
    const long long ctas = static_cast<long long>(a.N) * a.Hk, want = (8LL * kBandSms + ctas - 1) / ctas;
    return static_cast<int>(std::max<long long>(1, std::min<long long>(std::min<long long>(want, tiles), 64)));
}

template <typename T>
cudaError_t launch(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    const int splits = few_splits(a);
    const BandPart part = band_part(a, splits, ws);
    const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.N) * a.Hk * splits);
    cudaError_t e = a.D > 64 ? tc::allow_smem<few_kernel<T, 4>>() : tc::allow_smem<few_kernel<T, 2>>();
    if (e != cudaSuccess) return e;
    if (a.D > 64)
        few_kernel<T, 4><<<grid, kThreads, Cfg<4>::smem, stream>>>(a, splits, static_cast<T*>(out), lse, part);
    else
        few_kernel<T, 2><<<grid, kThreads, Cfg<2>::smem, stream>>>(a, splits, static_cast<T*>(out), lse, part);
    e = cudaGetLastError();
    if (e != cudaSuccess || splits == 1) return e;
    return launch_band_join(a, splits, part, 1.f, out, lse, stream);
}

}  // namespace

bool band_few_fits(const BandArgs& a) {
    return a.dtype != 0 && static_cast<long long>(a.Lq) * a.G <= kRows && band_most_keys(a) > kBandExactKeys;
}
size_t band_few_part_bytes(const BandArgs& a) { return band_part_bytes(a, few_splits(a)); }
cudaError_t launch_band_few(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    return a.dtype == 1 ? launch<__half>(a, out, lse, ws, stream) : launch<__nv_bfloat16>(a, out, lse, ws, stream);
}

}  // namespace dcn4
