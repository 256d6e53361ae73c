// dcn4_band_fwd_tc.cu — the band attention's forward for 16-bit types on the
// fifth-generation tensor cores.
//
// One pass over the visible keys.  With t = log2(e) s (s the scaled, biased score)
// and a reference r that follows the running maximum of t,
//     p = 2^(t - r),  l = sum p,  o = sum p v,   out = o / l,  lse = ln 2 (r + log2 l).
// r is moved (and o, l rescaled) only when the maximum has outgrown it by 2^8: p
// then stays below 2^8, far inside fp16's range, and o, which lives in tensor
// memory, is almost never read back on the way.  p is rounded to the I/O type, the
// second product's operand; its sum is taken in fp32 before the rounding.
//
// A CTA holds two tiles of 128 rows (a row is a query of one of the heads that
// share a key head) and streams tiles of 128 keys past both, or, where a head has
// no more than one tile of rows, lets its two halves take the key tiles in turn.
// Warps 0-3 and 4-7 each own a tile's softmax (thread = row = TMEM lane), warps
// 8-11 fill operand tiles, one thread of warp 12 issues the MMAs:
//     S = Q K^T  (both operands in shared memory, 128 x 128 into tensor memory)
//     O += P V   (P written over S in tensor memory as 16-bit pairs)
// so that one tile's exponentials run under the other's products.  Of a key tile
// only the 32-column chunks that some row may see are computed; only chunks on the
// band's edge are masked element by element.
#include "dcn4_band_tc.cuh"

namespace dcn4 {
namespace {

using namespace tc;

constexpr int kThreads = 416, kProducer = 8, kMma = 12;
constexpr int kSlots = 4;             // ring of operand tiles: K, V, K, V
constexpr int kLag = 2;               // tiles of cp.async in flight behind the one being issued
constexpr float kRescale = 8.f;
constexpr int kTableExtra = 256;      // the bias table reaches this far past M: no clamp in a chunk that touches [-M, M]
constexpr int kTableBytes = 28 << 10;

// A bounded wait by a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t* mbar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait_or(smem_u32(mbar), parity, abort));
}

__device__ unsigned g_band_status;    // nonzero once a bounded wait gave up

// How rows map to tiles.
struct FwdShape {
    int pack;      // heads of a tile: G or 1
    int tq;        // queries of a tile: 128 / pack
    int alt;       // 1: one tile of rows, key tiles in turn; 0: two tiles of rows
    int blocks;    // CTAs along the queries
    int splits;    // CTAs along the keys
    int table;     // floats of one head's bias table
};

__host__ __device__ inline int table_floats(int M) { return 2 * (M + kTableExtra) + 1; }

// What a tile of rows sees of key tile `tile`: the chunks [ca, cb) of 32 keys; false if none.
struct RowBand {
    int plo, phi;  // positions of its live queries
    int lo, hi;    // keys of the window
    int sink;      // keys of the sinks
    bool any;
};
__device__ __forceinline__ RowBand row_band(const BandArgs& a, int start, int i0, int i1, int klen) {
    RowBand b;
    b.any = i0 <= i1;
    b.plo = start + i0;
    b.phi = start + i1;
    b.lo = max(0, b.plo - a.left);
    b.hi = min(klen, b.phi + a.right + 1);
    b.sink = min(a.sinks, b.hi);
    return b;
}
__device__ __forceinline__ bool chunks_of(const RowBand& b, int j0, int& ca, int& cb) {
    int lo = max(b.lo, j0), hi = min(b.hi, j0 + kTcRows);
    const int sink = min(b.sink, j0 + kTcRows);
    if (sink > j0) {
        if (lo >= hi) hi = sink;
        lo = j0;
    }
    ca = (lo - j0) / kTcChunk;
    cb = (hi - j0 + kTcChunk - 1) / kTcChunk;
    return b.any && lo < hi;
}

struct Row {           // a softmax thread's row
    int pos;           // position of its query
    int jlo, jhi;      // keys of its window
    float m, l;        // reference (log2 units without a bias, natural with one) and sum
};

// The scores of one chunk: raw products in x; masked ones become -infinity * sign.
__device__ __forceinline__ bool sees(const Row& r, int sinks, int j) { return j < r.jhi && (j >= r.jlo || j < sinks); }

template <typename T, int NB, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_kernel(BandArgs a, FwdShape sh, T* __restrict__ out, float* __restrict__ lse, BandPart part) {
    extern __shared__ __align__(1024) unsigned char band_smem[];
    __shared__ __align__(8) uint64_t full[kSlots], empty[kSlots], q_full, s_full[2], p_full[2], o_done[2];
    __shared__ uint32_t taddr_s;
    __shared__ int s_abort;
    __shared__ float2 s_ml[kTcRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(band_smem) + 1023u) & ~1023u;
    const uint32_t qs = base, ring = base + (sh.alt ? 1 : 2) * NB * kTcBlock;
    float* table = reinterpret_cast<float*>(band_smem + (ring - smem_u32(band_smem)) + kSlots * NB * kTcBlock);

    int b = blockIdx.x;
    const int sp = b % sh.splits;
    b /= sh.splits;
    const int blk = sh.blocks - 1 - b % sh.blocks;  // the longest rows of a causal band first
    b /= sh.blocks;
    const int groups = a.Hq / sh.pack, n = b / groups, grp = b - n * groups, h0 = grp * sh.pack, hk = h0 / a.G;
    const int klen = band_klen(a, n), qlen = band_qlen(a, n), start = band_start(a, n);
    const int tiles = sh.alt ? 1 : 2;
    const int i0 = blk * tiles * sh.tq, i1 = min(i0 + tiles * sh.tq, qlen) - 1;

    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 4);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&q_full), 4);
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&s_full[w]), 1);
            mbar_init(smem_u32(&p_full[w]), 4);
            mbar_init(smem_u32(&o_done[w]), 1);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) {  // S and O of both halves
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&taddr_s)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (BIAS) {  // the bias of every head of the tile by relative position
        for (int e = tid; e < sh.pack * sh.table; e += kThreads) {
            const int g = e / sh.table, rel = e - g * sh.table - a.M - kTableExtra;
            const int bk = __ldg(a.buckets + max(-a.M, min(rel, a.M)) + a.M);
            table[e] = static_cast<unsigned>(bk) < static_cast<unsigned>(a.nb)
                           ? to_f32(static_cast<const T*>(a.bias)[static_cast<long long>(bk) * a.Hq + h0 + g]) : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = taddr_s;
    volatile int* abort = &s_abort;

    int t0 = 0, t1 = 0;
    BandTiles bt{0, 0, 0};
    if (i0 <= i1) {
        bt = band_tiles(a, start + i0, start + i1, klen, kTcRows);
        const long long cnt = bt.count();
        t0 = static_cast<int>(cnt * sp / sh.splits);
        t1 = static_cast<int>(cnt * (sp + 1) / sh.splits);
    }
    auto band_of = [&](int w) {
        const int lo = i0 + w * sh.tq;
        return row_band(a, start, lo, min(lo + sh.tq, qlen) - 1, klen);
    };
    // whether half w works on key tile t, and on which chunks
    const RowBand rb0 = band_of(0), rb1 = sh.alt ? rb0 : band_of(1);
    auto active = [&](int w, int t, int& ca, int& cb) {
        if (t >= t1 || (sh.alt && ((t - t0) & 1) != w)) return false;
        return chunks_of(w ? rb1 : rb0, bt.tile(t) * kTcRows, ca, cb);
    };

    if (warp >= kProducer && warp < kMma) {
        const int pt = tid - kProducer * 32;
        const T* q = static_cast<const T*>(a.q) + n * a.q_batch + static_cast<long long>(h0) * a.D;
        const T* k = static_cast<const T*>(a.k) + n * a.k_batch + static_cast<long long>(hk) * a.D;
        const T* v = static_cast<const T*>(a.v) + n * a.v_batch + static_cast<long long>(hk) * a.D;
        for (int w = 0; w < tiles && t0 < t1; ++w)
            load_operand<T, NB>(qs + w * NB * kTcBlock, a.D, kTcRows, q, [&](int r) -> const T* {
                const int ql = r / sh.pack, i = i0 + w * sh.tq + ql;
                return ql < sh.tq && i < qlen ? q + i * a.q_row + static_cast<long long>(r - ql * sh.pack) * a.D : nullptr;
            }, pt);
        cp_commit();
        const int items = 2 * (t1 - t0);
        for (int it = 0; it < items + kLag; ++it) {
            if (it < items) {
                const int s = it % kSlots, j0 = bt.tile(t0 + (it >> 1)) * kTcRows;
                if (!warp_wait(&empty[s], ((it / kSlots) & 1) ^ 1u, abort)) break;
                const T* src = it & 1 ? v : k;
                const long long row = it & 1 ? a.v_row : a.k_row;
                load_operand<T, NB>(ring + s * NB * kTcBlock, a.D, kTcRows, src,
                                    [&](int r) -> const T* { return j0 + r < klen ? src + (j0 + r) * row : nullptr; }, pt);
            }
            cp_commit();
            if (it >= kLag) {
                cp_wait<kLag>();
                fence_async_smem();  // the tensor cores read through the async proxy
                __syncwarp();
                if (lane == 0) {
                    if (it == kLag) mbar_arrive(smem_u32(&q_full));
                    mbar_arrive(smem_u32(&full[(it - kLag) % kSlots]));
                }
            }
        }
        cp_wait<0>();
    } else if (warp == kMma) {
        if (lane == 0 && t0 < t1) {
            const int steps = (a.D + 15) / 16;
            const uint32_t id_o = umma_idesc<T>(kTcRows, steps * 16, 0, 1);
            bool ok = mbar_wait_or(smem_u32(&q_full), 0u, abort);
            auto slot = [&](int it) { return ring + (it % kSlots) * NB * kTcBlock; };
            auto wait_tile = [&](int it) {
                ok = ok && mbar_wait_or(smem_u32(&full[it % kSlots]), (it / kSlots) & 1, abort);
                tc_fence_after();
            };
            auto scores = [&](int w, int t, int ca, int cb) {
                const int it = 2 * (t - t0);
                wait_tile(it);
                if (!ok) return;
                issue_rows(tmem + w * 128 + ca * kTcChunk, qs + (sh.alt ? 0 : w) * NB * kTcBlock, slot(it) + ca * kTcChunk * 128,
                           umma_idesc<T>(kTcRows, (cb - ca) * kTcChunk, 0, 0), steps);
                umma_commit(smem_u32(&s_full[w]));
            };
            int nw[2] = {0, 0};
            int ca, cb;
            for (int w = 0; w < 2; ++w)
                if (ok && active(w, t0, ca, cb)) scores(w, t0, ca, cb);
            umma_commit(smem_u32(&empty[0]));
            for (int t = t0; t < t1 && ok; ++t) {
                bool now[2], next[2];
                int na[2], nb_[2], xa[2], xb[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    now[w] = active(w, t, na[w], nb_[w]);
                    next[w] = active(w, t + 1, xa[w], xb[w]);
                }
#pragma unroll
                for (int w = 0; w < 2; ++w)  // a half that rests on this tile starts on the next one
                    if (ok && !now[w] && next[w]) scores(w, t + 1, xa[w], xb[w]);
                const int iv = 2 * (t - t0) + 1;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (!now[w] || !ok) continue;
                    wait_tile(iv);
                    ok = ok && mbar_wait_or(smem_u32(&p_full[w]), nw[w] & 1, abort);
                    tc_fence_after();
                    if (!ok) break;
                    issue_sum(tmem + 256 + w * 64 * NB, tmem + w * 128, slot(iv), id_o, na[w] * 2, nb_[w] * 2, nw[w] > 0);
                    umma_commit(smem_u32(&o_done[w]));
                    ++nw[w];
                    if (next[w]) scores(w, t + 1, xa[w], xb[w]);  // its S takes P's place, after the product that reads P
                }
                if (!ok) break;
                if (!now[0] && !now[1]) wait_tile(iv);  // nobody reads this tile's values
                umma_commit(smem_u32(&empty[iv % kSlots]));
                if (t + 1 < t1) {
                    if (!next[0] && !next[1]) wait_tile(iv + 1);
                    umma_commit(smem_u32(&empty[(iv + 1) % kSlots]));
                }
            }
            if (*abort) {  // the MMAs already issued must end before the memory goes
                umma_commit(smem_u32(&q_full));
                int never = 0;
                mbar_wait_or(smem_u32(&q_full), 1u, &never);
            }
        }
        __syncwarp();
    } else if (warp < kProducer) {
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_at = lane_base + w * 128, o_at = lane_base + 256 + w * 64 * NB;
        const int ql = row / sh.pack, g = row - ql * sh.pack, i = i0 + (sh.alt ? 0 : w) * sh.tq + ql;
        const bool live = ql < sh.tq && i < qlen;
        const bool warp_live = __any_sync(0xffffffffu, live);
        const RowBand& rb = w ? rb1 : rb0;
        Row r;
        r.pos = start + i;
        r.jlo = max(0, r.pos - a.left);
        r.jhi = min(klen, r.pos + a.right + 1);
        r.m = -INFINITY;
        r.l = 0.f;
        const int sinks = a.sinks;
        const float sc = BIAS ? a.scale : a.scale * kLog2e;
        const bool neg = sc < 0.f;
        const float* tab = table + g * sh.table + a.M + kTableExtra - r.pos;
        int nw = 0, ca, cb;
        bool ok = true;
        for (int t = t0; t < t1; ++t) {
            if (!active(w, t, ca, cb)) continue;
            const int j0 = bt.tile(t) * kTcRows;
            ok = warp_wait(&s_full[w], nw & 1, abort);
            if (!ok) break;
            tc_fence_after();
            if (warp_live) {
                // every row sees every key of these chunks
                auto clear = [&](int c) { const int j = j0 + c * kTcChunk; return j + kTcChunk <= min(klen, rb.plo + a.right + 1) && j >= rb.phi - a.left; };
                // 0: each pair has its own bias; 1, -1: all are beyond M, ahead or behind
                auto side = [&](int c) { const int j = j0 + c * kTcChunk; return j - rb.phi >= a.M ? 1 : j + kTcChunk - 1 - rb.plo <= -a.M ? -1 : 0; };
                auto scored = [&](uint32_t (&x)[32], int c) {  // natural scores with their bias
                    const int j = j0 + c * kTcChunk, sd = side(c);
                    if (sd == 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), sc, tab[j + e]));
                    } else {
                        const float bb = table[g * sh.table + (sd > 0 ? sh.table - 1 : 0)];
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), sc, bb));
                    }
                };
                // the tile's maximum (of raw products without a bias: their minimum under a negative scale)
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto fold = [&](uint32_t (&x)[32], int c) {
                    if (BIAS) scored(x, c);
                    if (!clear(c)) {
                        const int j = j0 + c * kTcChunk;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!sees(r, sinks, j + e)) x[e] = __float_as_uint(!BIAS && neg ? INFINITY : -INFINITY);
                    }
                    if (!BIAS && neg) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], -__uint_as_float(x[e]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(x[e]));
                    }
                };
                uint32_t x[32], y[32];
                for (int c = ca; c < cb; c += 2) {
                    tmem_ld32_async(s_at + c * kTcChunk, x);
                    if (c + 1 < cb) tmem_ld32_async(s_at + (c + 1) * kTcChunk, y);
                    tmem_ld_wait(x);
                    fold(x, c);
                    if (c + 1 < cb) {
                        tmem_ld_wait(y);
                        fold(y, c + 1);
                    }
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (!BIAS && top != -INFINITY) top *= fabsf(sc);
                constexpr float unit = BIAS ? kLog2e : 1.f;  // of m, to log2
                if (nw == 0) {
                    r.m = top;
                } else if (__any_sync(0xffffffffu, (top - r.m) * unit > kRescale)) {
                    // a maximum outgrew its reference (or a row sees its first key): move the references
                    const float to = fmaxf(top, r.m);
                    const float f = to == -INFINITY ? 1.f : ex2((r.m - to) * unit);
                    r.m = to;
                    r.l *= f;
                    ok = warp_wait(&o_done[w], (nw - 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    for (int d = 0; d < a.D; d += 32) {
                        tmem_ld32_async(o_at + d, x);
                        tmem_ld_wait(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                        tmem_st32(o_at + d, x);
                    }
                }
                const float ref = r.m == -INFINITY ? 0.f : r.m;
                float sum[4] = {};
                auto probs = [&](uint32_t (&x)[32], int c) {
                    if (BIAS) {
                        scored(x, c);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(ex2((__uint_as_float(x[e]) - ref) * kLog2e));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(ex2(fmaf(__uint_as_float(x[e]), sc, -ref)));
                    }
                    if (!clear(c)) {
                        const int j = j0 + c * kTcChunk;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!sees(r, sinks, j + e)) x[e] = 0u;
                    }
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float lo = __uint_as_float(x[2 * e]), hi = __uint_as_float(x[2 * e + 1]);
                        sum[(2 * e) & 3] += lo;
                        sum[(2 * e + 1) & 3] += hi;
                        p[e] = pack2<T>(lo, hi);
                    }
                    tmem_st16(s_at + c * 16, p);  // over columns whose scores have been read
                };
                for (int c = ca; c < cb; c += 2) {
                    tmem_ld32_async(s_at + c * kTcChunk, x);
                    if (c + 1 < cb) tmem_ld32_async(s_at + (c + 1) * kTcChunk, y);
                    tmem_ld_wait(x);
                    if (c + 1 < cb) tmem_ld_wait(y);
                    probs(x, c);
                    if (c + 1 < cb) probs(y, c + 1);
                }
                r.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st_wait();
            }
            ++nw;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[w]));
        }
        if (ok && nw > 0) ok = warp_wait(&o_done[w], (nw - 1) & 1, abort);
        tc_fence_after();
        if (sh.alt) {
            // the second half's rows are the first's: join them (its O is in the same lanes)
            if (w == 1) s_ml[row] = make_float2(r.m, nw > 0 && warp_live ? r.l : 0.f);
            tc_fence_before();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            tc_fence_after();
        }
        const bool rows_here = ql < sh.tq && i < a.Lq;
        if (ok && !(sh.alt && w == 1) && __any_sync(0xffffffffu, rows_here)) {
            constexpr float unit = BIAS ? kLog2e : 1.f;
            float f0 = 1.f, f1 = 0.f, m = r.m, l = live ? r.l : 0.f;
            bool first = nw > 0, second = false;
            if (sh.alt) {
                const float2 other = s_ml[row];
                const float l1 = live ? other.y : 0.f;
                m = fmaxf(r.m, l1 > 0.f ? other.x : -INFINITY);
                const float ref = m == -INFINITY ? 0.f : m;
                f0 = l > 0.f ? ex2((r.m - ref) * unit) : 0.f;
                f1 = l1 > 0.f ? ex2((other.x - ref) * unit) : 0.f;
                l = l * f0 + l1 * f1;
                second = t1 - t0 > 1 && __any_sync(0xffffffffu, l1 > 0.f);
            }
            const float mn = BIAS ? m : m * kLn2;
            const long long at = (static_cast<long long>(n) * a.Hq + h0 + g) * a.Lq + i;
            const bool split = sh.splits > 1;
            const float inv = l > 0.f ? (split ? 1.f : 1.f / l) : 0.f;
            f0 = l > 0.f ? f0 * inv : 0.f;
            f1 *= inv;
            if (rows_here) {
                if (split)
                    part.ml[at * sh.splits + sp] = make_float2(l > 0.f ? mn : -INFINITY, l);
                else
                    lse[at] = l > 0.f ? mn + logf(l) : -INFINITY;
            }
            T* to = out + ((static_cast<long long>(n) * a.Lq + i) * a.Hq + h0 + g) * a.D;
            float* po = part.o + (at * sh.splits + sp) * a.D;
            for (int d = 0; d < a.D; d += 32) {
                uint32_t x[32], y[32];
                if (first) tmem_ld32_async(o_at + d, x);
                if (second) tmem_ld32_async(o_at + 64 * NB + d, y);
                if (first) tmem_ld_wait(x);
                if (second) tmem_ld_wait(y);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float o = first && f0 != 0.f ? __uint_as_float(x[e]) * f0 : 0.f;
                    if (second && f1 != 0.f) o = fmaf(__uint_as_float(y[e]), f1, o);
                    x[e] = __float_as_uint(o);
                }
                if (!rows_here) continue;
                if (split) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (d + e < a.D)
                            *reinterpret_cast<float4*>(po + d + e) = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]),
                                                                                 __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        if (d + e < a.D) {
                            uint4 u;
                            u.x = pack2<T>(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                            u.y = pack2<T>(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                            u.z = pack2<T>(__uint_as_float(x[e + 4]), __uint_as_float(x[e + 5]));
                            u.w = pack2<T>(__uint_as_float(x[e + 6]), __uint_as_float(x[e + 7]));
                            *reinterpret_cast<uint4*>(to + d + e) = u;
                        }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort) atomicOr(&g_band_status, 1u);
    if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

FwdShape shape_of(const BandArgs& a) {
    FwdShape s;
    s.table = a.nb ? table_floats(a.M) : 0;
    s.pack = a.G;
    if (s.pack * s.table * static_cast<int>(sizeof(float)) > kTableBytes) s.pack = 1;
    s.tq = kTcRows / s.pack;
    s.alt = a.Lq <= s.tq;
    s.blocks = s.alt ? 1 : (a.Lq + 2 * s.tq - 1) / (2 * s.tq);
    const long long ctas = static_cast<long long>(a.N) * (a.Hq / s.pack) * s.blocks;
    s.splits = band_splits(a, ctas, std::min(a.Lq, 2 * s.tq), kTcRows, 1);
    return s;
}

template <typename T, int NB, bool BIAS>
cudaError_t launch(const BandArgs& a, const FwdShape& s, void* out, float* lse, void* ws, cudaStream_t stream) {
    const size_t smem = 1024 + static_cast<size_t>((s.alt ? 1 : 2) + kSlots) * NB * kTcBlock + s.pack * s.table * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(fwd_kernel<T, NB, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const BandPart part = band_part(a, s.splits, ws);
    const long long ctas = static_cast<long long>(a.N) * (a.Hq / s.pack) * s.blocks * s.splits;
    fwd_kernel<T, NB, BIAS><<<static_cast<unsigned>(ctas), kThreads, smem, stream>>>(a, s, static_cast<T*>(out), lse, part);
    e = cudaGetLastError();
    if (e != cudaSuccess || s.splits == 1) return e;
    return launch_band_join(a, s.splits, part, out, lse, stream);
}

template <typename T>
cudaError_t launch_typed(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    const FwdShape s = shape_of(a);
    if (a.D > 64)
        return a.nb ? launch<T, 2, true>(a, s, out, lse, ws, stream) : launch<T, 2, false>(a, s, out, lse, ws, stream);
    return a.nb ? launch<T, 1, true>(a, s, out, lse, ws, stream) : launch<T, 1, false>(a, s, out, lse, ws, stream);
}

}  // namespace

size_t band_fwd_tc_part_bytes(const BandArgs& a) { return band_part_bytes(a, shape_of(a).splits); }

cudaError_t launch_band_fwd_tc(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    return a.dtype == 1 ? launch_typed<__half>(a, out, lse, ws, stream)
                        : launch_typed<__nv_bfloat16>(a, out, lse, ws, stream);
}

cudaError_t band_fwd_status(unsigned* status, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_band_status, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_band_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace dcn4
