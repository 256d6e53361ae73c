// dcn4_band_bwd_tc.cu — the band attention's backward for 16-bit types on the
// fifth-generation tensor cores: three kernels, no atomics.
//
//   stats     delta_i = <g_i, out_i> beside lse_i (+infinity for rows that see
//             nothing: their probabilities are then 0 without a mask).
//   grad_q    a CTA holds two tiles of 128 rows and streams tiles of 64 keys:
//             S = Q K^T, E = G V^T, d = p (E - delta), p = e^(S - lse), gq += d K.
//   grad_kv   a CTA holds 128 keys and streams tiles of 64 queries of every head
//             that shares them: S^T = K Q^T, E^T = V G^T, gv += p^T G, gk += d^T Q;
//             with a bias it also sums d along the diagonals (see there).
// Scores are recomputed by both kernels (7 products instead of 5): one kernel would
// have to add every gq from many CTAs, in an order that changes.
//
// out is rounded, so delta is off, by the same amount for all of a row's d.  The
// sum of a row's d is that error (it is 0 otherwise), so grad_q corrects delta by it
// for grad_kv, where it would add up: over the pairs of a bucket most of all.  For
// gq the error weighs as the mean of a row's keys, that is with the root of their
// number: a CTA of grad_q whose rows see at most kFewKeys goes over them twice and takes
// delta = sum p E from the first pass (one more pass of two of its three products; of
// a long causal band the first CTAs only, whose rows hold half of gq's norm).
//
// p and d go to the tensor cores as the I/O type (EXACT: as two numbers of it, see
// kBandExactKeys), over the scores they came from in
// tensor memory; the sums stay there in fp32 until they are rounded once.
//
// A row whose lse is far from 0 (band_far) gets its maximum and sum anew in grad_q's first
// pass; `weights`, 1 for all other rows, is the inverse of that sum for grad_kv.
//
// With a bias the tables of all heads that share a key head are held in shared memory;
// where they pass kTableBytes grad_q's tiles are of one head each, and grad_kv, which goes
// head by head, reloads the present head's.
//
// 2 x 4096 causal tokens, window 1024, 16 heads of 128 on 4: grad_q 129 us (its 90
// GFLOP at 700 TFLOP/s), grad_kv 158 us (120 GFLOP), stats 20 us, bound by MMAs of
// N = 64 from shared memory; 16 x 785 ragged tokens with a bias, 8 heads of 64: 80, 94
// and 10 us, bound by the latency of a step's chain (products, exponentials, products);
// 8 x 785 tokens, reach 128, 16 heads of 64: 98 and 135 us, on one key head 98 and 190.
#include "dcn4_band_tc.cuh"

namespace dcn4 {
namespace {

using namespace tc;

// Warps 0-15 form p and d, 16 loads, those from 17 on issue MMAs.  Two tiles of scores
// are in work at a time, and each has two warpgroups, a chunk of 32 columns each: the
// probabilities need no maximum, so chunks are independent (with one warpgroup a tile
// the SM's schedulers had two warps each to hide latencies with, and grad_kv of a
// 785 x 785 map with a bias took 124 us instead of 93).
constexpr int kProducer = 16, kMma = 17;
constexpr int kTile = 64;                              // keys or queries of a streamed tile: two chunks
constexpr int kTileBlock = kTile * 128;                // bytes of 64 of its columns
constexpr int kTableExtra = 160;                       // as in the forward: a chunk and a tile's rows past M
constexpr int kTableBytes = 28 << 10;
constexpr int kTmem = 512;
constexpr int kFewKeys = 512;

__device__ unsigned g_band_bwd_status;

__host__ __device__ inline int table_floats(int M) { return 2 * (M + kTableExtra) + 1; }
__host__ __device__ inline int padded_queries(int Lq) { return (Lq + kTile - 1) / kTile * kTile; }

// Bias of `heads` heads from h0 on by relative position, clamped; thread `at` of `threads`.
template <typename T>
__device__ __forceinline__ void fill_table(const BandArgs& a, float* table, int floats, int h0, int heads, int at, int threads) {
    for (int e = at; e < heads * floats; e += threads) {
        const int g = e / floats, rel = e - g * floats - a.M - kTableExtra;
        const int bk = __ldg(a.buckets + max(-a.M, min(rel, a.M)) + a.M);
        table[e] = static_cast<unsigned>(bk) < static_cast<unsigned>(a.nb)
                       ? to_f32(static_cast<const T*>(a.bias)[static_cast<long long>(bk) * a.Hq + h0 + g]) : 0.f;
    }
}

// (lse, delta) of every row, [N][Hq][padded Lq], and the weight of its probabilities
// (1; grad_q changes those of far rows).  Without a bias lse is in log2 units, as the
// scores are formed there.  `lanes` lanes a row, four rows a thread: bound by HBM.
template <typename T>
__global__ void __launch_bounds__(256) stats_kernel(BandArgs a, int lanes, const T* __restrict__ out, const float* __restrict__ lse,
                                                    const T* __restrict__ gout, float2* __restrict__ stats, float* __restrict__ weights) {
    constexpr int U = 4;
    const int LP = padded_queries(a.Lq), groups = 256 / lanes, blocks = (LP + groups * U - 1) / (groups * U);
    const int nh = blockIdx.x / blocks, n = nh / a.Hq, h = nh - n * a.Hq, i0 = (blockIdx.x - nh * blocks) * groups * U + threadIdx.x / lanes;
    const int piece = threadIdx.x % lanes, qlen = band_qlen(a, n);
    uint4 x[U], y[U];
    float l[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = i0 + u * groups;
        x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
        l[u] = INFINITY;
        if (i >= qlen) continue;
        const long long at = ((static_cast<long long>(n) * a.Lq + i) * a.Hq + h) * a.D + piece * 8;
        if (piece * 8 < a.D) {
            x[u] = __ldg(reinterpret_cast<const uint4*>(out + at));
            y[u] = __ldg(reinterpret_cast<const uint4*>(gout + at));
        }
        if (piece == 0) l[u] = band_lse_ref(lse[static_cast<long long>(nh) * a.Lq + i]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float2 p[4], q[4];
        unpack(x[u], p, T());
        unpack(y[u], q, T());
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) d = fmaf(p[e].x, q[e].x, fmaf(p[e].y, q[e].y, d));
        for (int o = lanes >> 1; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        const int i = i0 + u * groups;
        if (i < LP && piece == 0) {
            stats[static_cast<long long>(nh) * LP + i] = make_float2(a.nb ? l[u] : l[u] * kLog2e, d);
            weights[static_cast<long long>(nh) * LP + i] = 1.f;
        }
    }
}

// ---------------------------------------------------------------------------
// grad_q
// ---------------------------------------------------------------------------
template <int NB, bool BIAS>
struct QCfg {
    static constexpr int slots = NB == 1 ? 6 : BIAS ? 2 : 3;
    static constexpr int threads = (kMma + 2) * 32;  // an issuing warp a half
    static constexpr size_t smem = 1024 + 4 * NB * kTcBlock + slots * 2 * NB * kTileBlock;
};

// After a wait that gave up: the block's results are NaN (and through delta its rows' part in grad_kv), and the
// status word says so.  (A call, with nothing of the kernel's own, so that its registers are those of the way
// without it: as part of grad_kv it cost 5 %.)
template <typename T>
__device__ __noinline__ void q_gave_up(BandArgs a, int pack, int tq, int blocks, float2* stats, T* gq) {
    if (threadIdx.x == 0) atomicOr(&g_band_bwd_status, 1u);
    const int blk = blocks - 1 - blockIdx.x % blocks, b = blockIdx.x / blocks, groups = a.Hq / pack, n = b / groups, h0 = (b - n * groups) * pack;
    const int i0 = blk * 2 * tq, rows = max(min(i0 + 2 * tq, a.Lq) - i0, 0) * pack;
    for (int r = threadIdx.x; r < rows; r += blockDim.x) {
        const int i = i0 + r / pack, h = h0 + r % pack;
        fill_nan(&stats[(static_cast<long long>(n) * a.Hq + h) * padded_queries(a.Lq) + i].y, 1);
        fill_nan(gq + ((static_cast<long long>(n) * a.Lq + i) * a.Hq + h) * a.D, a.D);
    }
}

template <typename T, int NB, bool BIAS, bool EXACT>
__global__ void __launch_bounds__(QCfg<NB, BIAS>::threads, 1)
    grad_q_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_g,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, BandArgs a, int pack,
                  int tq, int blocks, int floats, float2* __restrict__ stats, float* __restrict__ weights,
                  int* __restrict__ far_blocks, T* __restrict__ gq) {
    constexpr int kSlots = QCfg<NB, BIAS>::slots;
    extern __shared__ __align__(1024) unsigned char band_smem[];
    __shared__ __align__(8) uint64_t full[kSlots], empty[kSlots], raw, rows_full, s_full[2], e_full[2], p_full[2], o_done[2], ahead;
    __shared__ uint32_t taddr_s;
    __shared__ int s_abort;
    __shared__ float s_off[2][kTcRows];  // the second chunk's part of a row's sum
    const int tid = threadIdx.x, warp = static_cast<int>(uniform(tid >> 5)), lane = tid & 31;
    const uint32_t base = (smem_u32(band_smem) + 1023u) & ~1023u;
    const uint32_t qs = base, ring = base + 4 * NB * kTcBlock;  // Q, G of the first half, then of the second
    float* table = reinterpret_cast<float*>(band_smem + (ring - smem_u32(band_smem)) + kSlots * 2 * NB * kTileBlock);

    int b = blockIdx.x;
    const int blk = blocks - 1 - b % blocks;
    b /= blocks;
    const int groups = a.Hq / pack, n = b / groups, h0 = (b - n * groups) * pack, hk = h0 / a.G;
    const int klen = static_cast<int>(uniform(band_klen(a, n))), qlen = static_cast<int>(uniform(band_qlen(a, n))),
              start = static_cast<int>(uniform(band_start(a, n)));
    const int i0 = blk * 2 * tq, i1 = min(i0 + 2 * tq, qlen) - 1;
    // the row of a softmax thread: of half w, and the chunk c of its columns
    const int w = (warp >> 2) & 1, c = warp >> 3, row = tid & 127, ql = row / pack, g = row - ql * pack, i = i0 + w * tq + ql;
    const bool live = warp < kProducer && ql < tq && i < qlen;
    const long long stat_of = (static_cast<long long>(n) * a.Hq + h0 + g) * padded_queries(a.Lq) + i;
    const float2 st = live ? stats[stat_of] : make_float2(INFINITY, 0.f);

    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 2);
        }
        mbar_init(smem_u32(&raw), 1);
        mbar_init(smem_u32(&rows_full), 1);
        mbar_init(smem_u32(&ahead), 8);
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&s_full[w]), 1);
            mbar_init(smem_u32(&e_full[w]), 1);
            mbar_init(smem_u32(&p_full[w]), 8);
            mbar_init(smem_u32(&o_done[w]), 1);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&taddr_s)), "r"(kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (BIAS) fill_table<T>(a, table, floats, h0, pack, tid, QCfg<NB, BIAS>::threads);
    tc_fence_before();
    const bool far = uniform(__syncthreads_or(band_far(st.x))) != 0;  // some row's sum is not in its lse
    tc_fence_after();
    const uint32_t tmem = uniform(taddr_s);
    volatile int* abort = &s_abort;

    BandTiles bt{0, 0, 0};
    if (i0 <= i1) bt = band_tiles(a, start + i0, start + i1, klen, kTile);
    if (tid == 0) far_blocks[(n * groups + h0 / pack) * blocks + blk] = far;
    // tiles to go over: with `twice`, first for delta alone (and for the rows' maxima and sums, where `far`)
    const int tiles = bt.count();
    const bool twice = tiles * kTile <= kFewKeys || far;
    const int first = twice ? tiles : 0, cnt = first + tiles;
    auto tile_at = [&](int t) { return bt.tile(t < first ? t : t - first) * kTile; };
    // what a half's rows see of key tile t: chunks [ca, cb)
    auto band_of = [&](int w, int& plo, int& phi) {
        plo = start + i0 + w * tq;
        phi = min(plo + tq, start + qlen) - 1;
    };
    auto active = [&](int w, int t, int& ca, int& cb) {
        int plo, phi;
        band_of(w, plo, phi);
        const int j0 = tile_at(t), end = min(klen, phi + a.right + 1), sink = min(min(a.sinks, end), j0 + kTile);
        int lo = max(max(0, plo - a.left), j0), hi = min(end, j0 + kTile);
        if (sink > j0) {
            if (lo >= hi) hi = sink;
            lo = j0;
        }
        ca = (lo - j0) >> 5;
        cb = (hi - j0 + kTcChunk - 1) >> 5;
        return plo <= phi && lo < hi;
    };

    if (warp == kProducer) {
        if (cnt && elect_one()) {
            mbar_expect_tx(smem_u32(&rows_full), 4 * NB * pack * tq * 128);
            for (int w = 0; w < 2; ++w)
                for (int c = 0; c < NB; ++c) {
                    tma_load_rows(qs + (2 * w * NB + c) * kTcBlock, &map_q, c * 64, h0, i0 + w * tq, n, smem_u32(&rows_full));
                    tma_load_rows(qs + ((2 * w + 1) * NB + c) * kTcBlock, &map_g, c * 64, h0, i0 + w * tq, n, smem_u32(&rows_full));
                }
        }
        int raws = 0;
        for (int t = 0; t < cnt; ++t) {
            const int s = t % kSlots, j0 = tile_at(t);
            if (!warp_wait(&empty[s], ((t / kSlots) & 1) ^ 1u, abort)) break;
            const uint32_t at_k = ring + s * 2 * NB * kTileBlock, at_v = at_k + NB * kTileBlock;
            const bool clear = j0 + kTile > klen && klen < a.Lk;  // keys past the sequence meet d of 0
            if (elect_one()) {
                const uint32_t bar = smem_u32(clear ? &raw : &full[s]);
                mbar_expect_tx(bar, 2 * NB * kTileBlock);
                for (int c = 0; c < NB; ++c) {
                    tma_load_rows(at_k + c * kTileBlock, &map_k, c * 64, hk, j0, n, bar);
                    tma_load_rows(at_v + c * kTileBlock, &map_v, c * 64, hk, j0, n, bar);
                }
            }
            if (clear) {
                if (!warp_wait(&raw, raws++ & 1, abort)) break;
                zero_rows<2 * NB>(at_k, kTileBlock, max(klen - j0, 0), kTile, lane);
                if (elect_one()) mbar_arrive(smem_u32(&full[s]));
            }
        }
    } else if (warp >= kMma) {
        const int w = warp - kMma;
        if (cnt) {
            const int steps = (a.D + 15) / 16;
            const uint32_t id_s = umma_idesc<T>(kTcRows, 0, 0, 0), id_o = umma_idesc<T>(kTcRows, steps * 16, 0, 1);
            const uint64_t q_desc = umma_desc_sw128(qs + 2 * w * NB * kTcBlock, 16, 1024), g_desc = step_desc(q_desc, NB * kTcBlock),
                           k_desc = umma_desc_sw128(ring, 16, 1024), v_desc = step_desc(k_desc, NB * kTileBlock),
                           k_sum = umma_desc_sw128(ring, kTileBlock, 1024);
            const uint32_t at_s = tmem + w * 256, at_o = at_s + 128;
            bool ok = warp_wait(&rows_full, 0u, abort), some = false;
            uint32_t p_phase = 0;
            // half a step behind the first half, so that one's products run under the other's exponentials
            // (a barrier that completes once: p_full would go on without this warp, and its parity come round)
            int ca0, cb0;
            if (w == 1 && active(0, 0, ca0, cb0)) ok = ok && warp_wait(&ahead, 0u, abort);
            int s = 0;
            uint32_t ph = 0;
#pragma unroll 1
            for (int t = 0; t < cnt && ok; ++t) {
                int ca, cb;
                const bool on = active(w, t, ca, cb);
                if (!(ok = warp_wait(&full[s], ph, abort))) break;
                tc_fence_after();
                const uint32_t off = s * 2 * NB * kTileBlock, row = off + ca * kTcChunk * 128;
                if (on) {
                    if (elect_one()) {
                        const uint32_t id = id_s | (static_cast<uint32_t>((cb - ca) * (kTcChunk / 8)) << 17);
                        issue_rows<NB>(at_s + ca * kTcChunk, q_desc, kTcBlock, step_desc(k_desc, row), kTileBlock, id, steps);
                        umma_commit(smem_u32(&s_full[w]));  // the exponentials run under the second product
                        issue_rows<NB>(at_s + 64 + ca * kTcChunk, g_desc, kTcBlock, step_desc(v_desc, row), kTileBlock, id, steps);
                        umma_commit(smem_u32(&e_full[w]));
                    }
                    __syncwarp();
                    if (!(ok = warp_wait(&p_full[w], p_phase, abort))) break;
                    tc_fence_after();
                    p_phase ^= 1u;
                    if (t >= first) {
                        if (elect_one()) {
                            issue_sum<kTile / 16>(at_o, at_s, step_desc(k_sum, off), id_o, ca * 2, cb * 2, some);
                            if (EXACT) issue_sum<kTile / 16>(at_o, at_s + kLow, step_desc(k_sum, off), id_o, ca * 2, cb * 2, true);
                        }
                        __syncwarp();
                        some = true;
                    }
                }
                if (elect_one()) umma_commit(smem_u32(&empty[s]));
                __syncwarp();
                s = s + 1 == kSlots ? 0 : s + 1;
                ph ^= s == 0;
            }
            if (elect_one()) umma_commit(smem_u32(&o_done[w]));
            __syncwarp();
            int never = 0;
            if (!ok && lane == 0) mbar_wait_or(smem_u32(&o_done[w]), 0u, &never);  // the MMAs must end before the memory goes
        }
        __syncwarp();
    } else if (warp < kProducer) {
        const uint32_t at_h = tmem + w * 256 + (static_cast<uint32_t>((warp & 3) * 32) << 16), at_s = at_h + c * kTcChunk, at_o = at_h + 128;
        const bool warp_live = __any_sync(0xffffffffu, live);
        int plo, phi;
        band_of(w, plo, phi);
        const int pos = start + i;
        const int jlo = max(0, pos - a.left), jhi = min(klen, pos + a.right + 1), jsink = min(a.sinks, jhi);
        const int all_lo = phi - a.left, all_hi = min(klen, plo + a.right + 1) - kTcChunk;  // keys that all rows of the tile see
        // p = 2^(score - ref) * weight; off: the sum of the row's d, or in the first pass of p E
        float ref = st.x, weight = 1.f, delta = twice ? 0.f : st.y, shift = -delta, off = 0.f;
        const float sc = BIAS ? a.scale : a.scale * kLog2e;
        const float* tab = table + g * floats + a.M + kTableExtra - pos;
        // the row's sum (or maximum) over both chunks, for the first chunk's thread (and, with `back`, the second's).
        // Each word is read by the other chunk's thread only, before a barrier that its next writer passes later.
        auto both = [&](float v, bool back, bool largest = false) {
            if (c) s_off[w][row] = v;
            asm volatile("bar.sync %0, 256;" ::"r"(1 + w) : "memory");
            if (!c) v = largest ? fmaxf(v, s_off[w][row]) : v + s_off[w][row];
            if (back) {
                if (!c) s_off[w][row] = v;
                asm volatile("bar.sync %0, 256;" ::"r"(1 + w) : "memory");
                if (c) v = s_off[w][row];
            }
            return v;
        };
        int nw = 0, ca, cb;
        bool ok = true;
        int t = 0;
        if (far) {
            // The first pass of a CTA with far rows: their maxima, sums and delta, as the forward forms them.  (In
            // sixteen columns at a time and beside the loop below, whose registers it would not leave alone.)
            float top = -INFINITY, sum = 0.f;
            constexpr float unit = BIAS ? kLog2e : 1.f;
            for (; t < first && ok; ++t) {
                if (!active(w, t, ca, cb)) continue;
                const int j = tile_at(t) + c * kTcChunk;
                ok = warp_wait(&s_full[w], nw & 1, abort) && warp_wait(&e_full[w], nw & 1, abort);
                tc_fence_after();
                if (ok && warp_live && c >= ca && c < cb) {
                    const uint32_t see = (low_bits(jhi - j) & ~low_bits(jlo - j)) | low_bits(jsink - j);
#pragma unroll 1
                    for (int h = 0; h < kTcChunk; h += 16) {
                        uint32_t x[16], y[16];
                        tmem_ld16(at_s + h, x);
                        tmem_ld16(at_s + 64 + h, y);
                        float most = top;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float s = __uint_as_float(x[e]);
                            if (BIAS) x[e] = __float_as_uint(fmaf(s, sc, tab[max(pos - a.M, min(j + h + e, pos + a.M))]));
                            if (see >> (h + e) & 1u) most = fmaxf(most, BIAS ? __uint_as_float(x[e]) : s * sc);
                        }
                        const float f = top == -INFINITY ? 0.f : ex2((top - most) * unit);
                        sum *= f;
                        off *= f;
                        top = most;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (!(see >> (h + e) & 1u)) continue;
                            const float s = __uint_as_float(x[e]), p = top == -INFINITY ? 0.f : ex2(BIAS ? (s - top) * unit : fmaf(s, sc, -top));
                            sum += p;
                            off = fmaf(p, __uint_as_float(y[e]), off);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&p_full[w]));
                    if (w == 0 && t == 0) mbar_arrive(smem_u32(&ahead));
                }
                ++nw;
            }
            t = first;
            ref = both(top, true, true);
            const float f = top == -INFINITY ? 0.f : ex2((top - ref) * unit), l = both(sum * f, true);
            off *= f;
            weight = l != 0.f ? 1.f / l : 1.f;
            ref = l != 0.f ? ref : INFINITY;
        }
        for (; t < cnt; ++t) {
            if (t == first && twice) {  // (also by a warp whose wait gave up: the others' barrier counts it)
                delta = both(off, true) * weight;
                shift = -delta * weight;
                off = 0.f;
            }
            if (!ok || !active(w, t, ca, cb)) continue;
            const int j = tile_at(t) + c * kTcChunk;
            const bool on = warp_live && c >= ca && c < cb;
            uint32_t x[32];
            ok = warp_wait(&s_full[w], nw & 1, abort);
            if (ok && on) {
                tc_fence_after();
                tmem_ld32_async(at_s, x);
                tmem_ld_wait(x);
                if (BIAS) {
                    const int side = j - phi >= a.M ? 1 : j + kTcChunk - 1 - plo <= -a.M ? -1 : 0;
                    if (side) {
                        const float bb = table[g * floats + (side > 0 ? floats - 1 : 0)];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) fma2(x[e], x[e + 1], sc, bb);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), sc, tab[j + e]));
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) sub_mul2(x[e], x[e + 1], ref, kLog2e);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) fma2(x[e], x[e + 1], sc, -ref);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(ex2(__uint_as_float(x[e])));
            }
            ok = ok && warp_wait(&e_full[w], nw & 1, abort);
            if (ok && on) {
                tc_fence_after();
                uint32_t y[32];
                tmem_ld32_async(at_s + 64, y);
                tmem_ld_wait(y);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * fmaf(__uint_as_float(y[e]), weight, shift));
                if (j < all_lo || j > all_hi) {
                    const uint32_t see = (low_bits(jhi - j) & ~low_bits(jlo - j)) | low_bits(jsink - j);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(see & (1u << e))) x[e] = 0u;
                }
                float2 sum[2] = {};
#pragma unroll
                for (int e = 0; e < 32; e += 2) add2(sum[(e >> 1) & 1], x[e], x[e + 1]);
                off += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (t >= first) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[e] = pack2<T>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                    tmem_st16(at_s, p);
                    if (EXACT) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = pack_low<T>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), p[e]);
                        tmem_st16(at_s + kLow, p);
                    }
                    tmem_st_wait();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&p_full[w]));
                if (w == 0 && t == 0) mbar_arrive(smem_u32(&ahead));
            }
            ++nw;
        }
        off = both(off, false);
        if (ok && live && !c) {
            stats[stat_of] = make_float2(ref, delta + off);
            if (far) weights[stat_of] = weight;
        }
        if (ok && cnt) ok = warp_wait(&o_done[w], 0u, abort);
        tc_fence_after();
        const bool rows_here = ql < tq && i < a.Lq;
        if (ok && __any_sync(0xffffffffu, rows_here)) {
            T* to = gq + ((static_cast<long long>(n) * a.Lq + i) * a.Hq + h0 + g) * a.D;
            for (int d = 32 * c; d < a.D; d += 64) {
                uint32_t x[32];
                if (nw) {
                    tmem_ld32_async(at_o + d, x);
                    tmem_ld_wait(x);
                }
                if (!rows_here) continue;
                const bool zero = !nw || !live;
#pragma unroll
                for (int e = 0; e < 32; e += 8)
                    if (d + e < a.D) {
                        uint32_t u[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            u[f] = zero ? 0u : pack2<T>(__uint_as_float(x[e + 2 * f]) * a.scale, __uint_as_float(x[e + 2 * f + 1]) * a.scale);
                        *reinterpret_cast<uint4*>(to + d + e) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort) q_gave_up<T>(a, pack, tq, blocks, stats, gq);
    if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
}

// ---------------------------------------------------------------------------
// grad_k and grad_v
// ---------------------------------------------------------------------------
// Items of an image and key head: every tile of 128 keys in `others` parts along the
// queries, those of the sinks (which see far more queries than the window) in `sinks`.
struct KvShape {
    int tiles, sink_tiles;
    int sink_parts, other_parts;
    int floats;             // of a head's bias table
    int whole;              // items of a key head that leave no parts, its last ones: all but the sinks', or none
    __host__ __device__ int items() const { return sink_tiles * sink_parts + (tiles - sink_tiles) * other_parts; }
    __host__ __device__ bool split() const { return sink_parts > 1 || other_parts > 1; }
};

// Diagonal sums.  All pairs of a diagonal of the score matrix share a relative
// position, so the bias gradient is the sum of d along diagonals, then over the
// diagonals of a bucket.  A warp's lanes hold keys; a chunk of 32 queries goes, in two
// halves, through 32 rows of 17 floats of shared memory and comes back by diagonals:
// lane k adds those of key - query = k and, apart, of k - 32, and each ends in one store
// of 32 neighbouring relative positions.  A warp meets every second chunk of 32 queries at
// most, so that no two of its stores meet: no atomics, one order.  (Handing partial
// sums from lane to lane needs no shared memory, but is a chain of 32 shuffles: 900
// cycles a chunk instead of 250.)
constexpr int kDiagBuf = 32 * 17;
constexpr int kDiagWarps = 16;  // sums a CTA leaves
struct Diagonals {
    float* mine;    // this warp's sums, of relative position -M .. M (the ends: and beyond)
    float* buf;     // this warp's kDiagBuf floats
    int M, rel0;    // relative position of lane 0's key and query 0
    float below, above;
    __device__ __forceinline__ void start(float* to) {
        mine = to;
        below = above = 0.f;
    }
    __device__ __forceinline__ void store(int rel, float v) {
        if (rel <= -M) below += v;
        else if (rel >= M) above += v;
        else mine[rel + M] = v;
    }
    __device__ __forceinline__ void chunk(int i, int lane, const uint32_t (&d)[32]) {
        float a[2] = {}, b[2] = {};  // of the halves: key - query of the half = lane, and lane - 32
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int e = 0; e < 16; ++e) buf[lane * 17 + e] = __uint_as_float(d[16 * z + e]);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = (lane + e) & 31;
                const float v = buf[r * 17 + e];
                if (r >= e) a[z] += v;
                else b[z] += v;
            }
            __syncwarp();
        }
        // the second half's queries are 16 later
        const float a1 = __shfl_xor_sync(0xffffffffu, a[1], 16), b1 = __shfl_xor_sync(0xffffffffu, b[1], 16);
        if (lane < 16) a[0] += a1, b[0] += b1;
        else b[0] += a1;
        store(rel0 - i + lane, a[0]);
        store(rel0 - i + lane - 32, b[0]);  // (lane 0's is an empty sum)
    }
    __device__ __forceinline__ void finish(int lane) {
        for (int o = 16; o; o >>= 1) {
            below += __shfl_xor_sync(0xffffffffu, below, o);
            above += __shfl_xor_sync(0xffffffffu, above, o);
        }
        if (lane == 0) {
            mine[0] = below;
            mine[2 * M] = above;
        }
    }
};

template <int NB, bool BIAS>
struct KvCfg {
    static constexpr int slots = NB == 1 ? 6 : BIAS ? 3 : 4;
    static constexpr int threads = (kMma + 1) * 32;
    static constexpr int stage = 2 * NB * kTileBlock;      // Q, G
    static constexpr int stat = kTile * sizeof(float2);
    static constexpr size_t smem = 1024 + 2 * NB * kTcBlock + slots * (stage + stat) + (BIAS ? kDiagWarps * kDiagBuf * sizeof(float) : 0);
};

// fill_table of one head by 256 threads (a call: its loop would take registers of the loop around it).
template <typename T>
__device__ __noinline__ void fill_head(BandArgs a, float* table, int floats, int h, int at) {
    fill_table<T>(a, table, floats, h, 1, at, 256);
}

// As q_gave_up.
template <typename T>
__device__ __noinline__ void kv_gave_up(BandArgs a, KvShape sh, T* gk, T* gv, float* part, float* diag) {
    if (threadIdx.x == 0) atomicOr(&g_band_bwd_status, 1u);
    const int items = sh.items(), nh = blockIdx.x / items, item = blockIdx.x - nh * items, n = nh / a.Hk, hk = nh - n * a.Hk;
    const int sink_items = sh.sink_tiles * sh.sink_parts;
    const bool is_sink = item < sink_items;
    const int parts = is_sink ? sh.sink_parts : sh.other_parts;
    const int k0 = (is_sink ? item / parts : sh.sink_tiles + (item - sink_items) / parts) * kTcRows;
    for (int r = threadIdx.x; r < kTcRows; r += blockDim.x) {
        for (int w = 0; w < 2 && parts > 1; ++w) fill_nan(part + ((static_cast<long long>(blockIdx.x - nh * sh.whole) * 2 + w) * kTcRows + r) * a.D, a.D);
        if (parts > 1 || k0 + r >= a.Lk) continue;
        const long long at = ((static_cast<long long>(n) * a.Lk + k0 + r) * a.Hk + hk) * a.D;
        fill_nan(gk + at, a.D);
        fill_nan(gv + at, a.D);
    }
    if (diag && threadIdx.x == 0) fill_nan(diag + static_cast<long long>(blockIdx.x) * kDiagWarps * a.G * (2 * a.M + 1), a.G * (2 * a.M + 1));
}

// WHOLE: the bias tables of all heads that share the key head are held at once; otherwise each parity holds its
// present head's and reloads it at the next (as a branch in one kernel that cost the others 18 %).
template <typename T, int NB, bool BIAS, bool EXACT, bool WHOLE>
__global__ void __launch_bounds__(KvCfg<NB, BIAS>::threads, 1)
    grad_kv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_g,
                   const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, BandArgs a, KvShape sh,
                   const float2* __restrict__ stats, const float* __restrict__ weights, const int* __restrict__ far_blocks,
                   int blocks, T* __restrict__ gk, T* __restrict__ gv,
                   float* __restrict__ part, float* __restrict__ diag) {
    using C = KvCfg<NB, BIAS>;
    constexpr int kSlots = C::slots;
    extern __shared__ __align__(1024) unsigned char band_smem[];
    __shared__ __align__(8) uint64_t full[kSlots], empty[kSlots], raw, keys_full, s_full[2], e_full[2], p_full[2], done;
    __shared__ uint32_t taddr_s;
    __shared__ int s_abort, s_part;  // s_part: this block's place among those that leave parts (formed where it is used it cost 3 %)
    const int tid = threadIdx.x, warp = static_cast<int>(uniform(tid >> 5)), lane = tid & 31;
    const uint32_t base = (smem_u32(band_smem) + 1023u) & ~1023u;
    const uint32_t ks = base, ring = base + 2 * NB * kTcBlock, stat_at = ring + kSlots * C::stage;
    const float4* stat_s = reinterpret_cast<const float4*>(band_smem + (stat_at - smem_u32(band_smem)));
    float* diag_s = reinterpret_cast<float*>(band_smem + (stat_at - smem_u32(band_smem)) + kSlots * C::stat);
    float* table = diag_s + (BIAS ? kDiagWarps * kDiagBuf : 0);

    const int items = sh.items(), nh = blockIdx.x / items, item = blockIdx.x - nh * items;
    const int n = nh / a.Hk, hk = nh - n * a.Hk;
    const int sink_items = sh.sink_tiles * sh.sink_parts;
    const bool is_sink = item < sink_items;
    const int parts = is_sink ? sh.sink_parts : sh.other_parts;
    const int rest = is_sink ? item : item - sink_items, kt = (is_sink ? 0 : sh.sink_tiles) + rest / parts, prt = rest % parts;
    const int k0 = kt * kTcRows;
    const int klen = static_cast<int>(uniform(band_klen(a, n))), qlen = static_cast<int>(uniform(band_qlen(a, n))),
              start = static_cast<int>(uniform(band_start(a, n)));
    const int k1 = min(k0 + kTcRows, klen);
    int ilo = 0, ihi = 0;
    if (k0 < klen) band_queries(a, start, qlen, k0, k1, ilo, ihi);
    const int q0 = ilo / kTile, nq = ilo < ihi ? (ihi - 1) / kTile - q0 + 1 : 0;
    const long long total = static_cast<long long>(nq) * a.G;
    const int t0 = static_cast<int>(total * prt / parts), cnt = static_cast<int>(total * (prt + 1) / parts) - t0;

    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&raw), 1);
        mbar_init(smem_u32(&keys_full), 1);
        mbar_init(smem_u32(&done), 1);
        s_part = blockIdx.x - nh * sh.whole;
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&s_full[w]), 1);
            mbar_init(smem_u32(&e_full[w]), 1);
            mbar_init(smem_u32(&p_full[w]), 8);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&taddr_s)), "r"(kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (BIAS && WHOLE) fill_table<T>(a, table, sh.floats, hk * a.G, a.G, tid, C::threads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(taddr_s);
    volatile int* abort = &s_abort;
    // step t: queries [tile * 64, + 64) of head hk G + g, of which the chunks [ca, cb) are in [ilo, ihi)
    // (even steps go through the first half of them, odd ones through the second: each softmax
    // half then meets neighbouring tiles)
    const int half = (cnt + 1) >> 1;
    struct Step {  // goes through every other step with additions only
        int g, r, nq;
        __device__ __forceinline__ Step(int u, int nq) : nq(nq) {
            g = nq ? u / nq : 0;
            r = u - g * nq;
        }
        __device__ __forceinline__ void next() {
            if (++r == nq) r = 0, ++g;
        }
    };
    auto first_of = [&](int odd) { return Step(t0 + (odd ? half : 0), nq); };
    auto chunks = [&](int i, int& ca, int& cb) {
        ca = (max(ilo, i) - i) >> 5;
        cb = (min(ihi, i + kTile) - i + kTcChunk - 1) >> 5;
    };

    if (warp == kProducer) {
        if (cnt && elect_one()) {
            mbar_expect_tx(smem_u32(&keys_full), 2 * NB * kTcBlock);
            for (int c = 0; c < NB; ++c) {
                tma_load_rows(ks + c * kTcBlock, &map_k, c * 64, hk, k0, n, smem_u32(&keys_full));
                tma_load_rows(ks + (NB + c) * kTcBlock, &map_v, c * 64, hk, k0, n, smem_u32(&keys_full));
            }
        }
        int raws = 0;
        const int LP = padded_queries(a.Lq);
        Step even = first_of(0), odd = first_of(1);
        for (int t = 0; t < cnt; ++t) {
            const int s = t % kSlots;
            const int g = t & 1 ? odd.g : even.g, i = (q0 + (t & 1 ? odd.r : even.r)) * kTile;
            if (t & 1) odd.next(); else even.next();
            if (!warp_wait(&empty[s], ((t / kSlots) & 1) ^ 1u, abort)) break;
            const uint32_t at_q = ring + s * C::stage, at_g = at_q + NB * kTileBlock;
            const bool clear = i + kTile > qlen && qlen < a.Lq;  // queries past the sequence meet p and d of 0
            if (elect_one()) {
                const uint32_t bar = smem_u32(clear ? &raw : &full[s]);
                mbar_expect_tx(bar, C::stage + C::stat);
                for (int c = 0; c < NB; ++c) {
                    tma_load_rows(at_q + c * kTileBlock, &map_q, c * 64, hk * a.G + g, i, n, bar);
                    tma_load_rows(at_g + c * kTileBlock, &map_g, c * 64, hk * a.G + g, i, n, bar);
                }
                const float2* src = stats + (static_cast<long long>(n) * a.Hq + hk * a.G + g) * LP + i;
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 stat_at + s * C::stat), "l"(src), "r"(C::stat), "r"(bar) : "memory");
            }
            if (clear) {
                if (!warp_wait(&raw, raws++ & 1, abort)) break;
                zero_rows<2 * NB>(at_q, kTileBlock, max(qlen - i, 0), kTile, lane);
                if (elect_one()) mbar_arrive(smem_u32(&full[s]));
            }
        }
    } else if (warp == kMma) {
        if (cnt) {
            const int steps = (a.D + 15) / 16;
            const uint32_t id_s = umma_idesc<T>(kTcRows, 0, 0, 0), id_o = umma_idesc<T>(kTcRows, steps * 16, 0, 1);
            const uint64_t k_desc = umma_desc_sw128(ks, 16, 1024), v_desc = step_desc(k_desc, NB * kTcBlock),
                           q_desc = umma_desc_sw128(ring, 16, 1024), g_desc = step_desc(q_desc, NB * kTileBlock),
                           q_sum = umma_desc_sw128(ring, kTileBlock, 1024), g_sum = step_desc(q_sum, NB * kTileBlock);
            bool ok = warp_wait(&keys_full, 0u, abort);
            int s = 0, sum_slot = 0;   // slots of steps t + 2 and t
            uint32_t ph = 0;
            Step even = first_of(0), odd = first_of(1);
            int span0 = 0, span1 = 0;  // chunks ca | cb << 8 of the even and the odd step in work
#pragma unroll 1
            for (int t = -2; t < cnt && ok; ++t) {
                const int z = t & 1;
                const bool more = t + 2 < cnt;
                int span = 0;
                if (more) {  // all of the next step that needs no wait for this one
                    int ca, cb;
                    chunks((q0 + (z ? odd.r : even.r)) * kTile, ca, cb);
                    if (z) odd.next(); else even.next();
                    span = ca | cb << 8;
                    if (!(ok = warp_wait(&full[s], ph, abort))) break;
                }
                const uint32_t at = tmem + z * 128;
                if (t >= 0) {
                    const int ca = (z ? span1 : span0) & 255, cb = (z ? span1 : span0) >> 8;
                    if (!(ok = warp_wait(&p_full[z], (t >> 1) & 1, abort))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t off = sum_slot * C::stage;
                        issue_sum<kTile / 16>(tmem + 256, at, step_desc(g_sum, off), id_o, ca * 2, cb * 2, t > 0);
                        issue_sum<kTile / 16>(tmem + 256 + 64 * NB, at + 64, step_desc(q_sum, off), id_o, ca * 2, cb * 2, t > 0);
                        if (EXACT) {
                            issue_sum<kTile / 16>(tmem + 256, at + kLow, step_desc(g_sum, off), id_o, ca * 2, cb * 2, true);
                            issue_sum<kTile / 16>(tmem + 256 + 64 * NB, at + 64 + kLow, step_desc(q_sum, off), id_o, ca * 2, cb * 2, true);
                        }
                        umma_commit(smem_u32(&empty[sum_slot]));
                    }
                    __syncwarp();
                    sum_slot = sum_slot + 1 == kSlots ? 0 : sum_slot + 1;
                }
                if (more) {  // over the place of p and d of step t
                    tc_fence_after();
                    if (elect_one()) {
                        const int ca = span & 255, cb = span >> 8;
                        const uint32_t off = s * C::stage + ca * kTcChunk * 128, to = at + ca * kTcChunk,
                                       id = id_s | (static_cast<uint32_t>((cb - ca) * (kTcChunk / 8)) << 17);
                        issue_rows<NB>(to, k_desc, kTcBlock, step_desc(q_desc, off), kTileBlock, id, steps);
                        umma_commit(smem_u32(&s_full[z]));  // the exponentials run under the second product
                        issue_rows<NB>(to + 64, v_desc, kTcBlock, step_desc(g_desc, off), kTileBlock, id, steps);
                        umma_commit(smem_u32(&e_full[z]));
                    }
                    __syncwarp();
                    (z ? span1 : span0) = span;
                    s = s + 1 == kSlots ? 0 : s + 1;
                    ph ^= s == 0;
                }
            }
            if (elect_one()) umma_commit(smem_u32(&done));
            __syncwarp();
            int never = 0;
            if (!ok && lane == 0) mbar_wait_or(smem_u32(&done), 0u, &never);
        }
        __syncwarp();
    } else {
        const int w = (warp >> 2) & 1, c = warp >> 3, row = tid & 127, j = k0 + row;  // steps of parity w, their chunk c
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t at_s = lane_base + w * 128 + c * kTcChunk;
        const bool warp_live = k0 + (warp & 3) * 32 < klen;
        // queries that see this key
        const int vlo = j - a.right - start, vhi = j >= klen ? 0 : j < a.sinks ? qlen : min(qlen, j + a.left - start + 1);
        // queries that see every key of the tile (with a bias a dead key's d must be 0, so its tile is masked)
        const int all_lo = BIAS && k1 - k0 < kTcRows ? kBandFar : k1 - 1 - a.right - start, all_hi = (k1 <= a.sinks ? qlen : min(qlen, k0 + a.left - start + 1)) - kTcChunk;
        const float sc = BIAS ? a.scale : a.scale * kLog2e;
        // whether some row of this key head is far (`blocks` of grad_q's CTAs went over them)
        int some = 0;
        for (int e = lane; e < blocks; e += 32) some |= far_blocks[nh * blocks + e];
        const bool far = __any_sync(0xffffffffu, some);
        const int kw = k0 + (warp & 3) * 32;  // this warp's keys
        Diagonals dg;
        int dg_head = -1, tab_head = -1;
        float* diag_w = diag + (static_cast<long long>(blockIdx.x) * kDiagWarps + warp) * a.G * (2 * a.M + 1);
        const bool sums = BIAS && diag;
        if (sums) {  // what no store below reaches is 0
            for (int e = lane; e < a.G * (2 * a.M + 1); e += 32) diag_w[e] = 0.f;
            __syncwarp();
        }
        dg.M = a.M;
        dg.rel0 = kw - start;
        dg.buf = diag_s + warp * kDiagBuf;
        bool ok = true;
        int s = w;
        Step st_w = first_of(w);
        for (int t = w; t < cnt; t += 2) {
            int ca, cb;
            const int g = st_w.g, i = (q0 + st_w.r) * kTile, ic = i + c * kTcChunk;
            st_w.next();
            if (!WHOLE && g != tab_head) {  // (also by a warp whose wait gave up: the others' barriers count it)
                asm volatile("bar.sync %0, 256;" ::"r"(1 + w) : "memory");  // the last head's reads are done
                fill_head<T>(a, table + w * sh.floats, sh.floats, hk * a.G + g, c * kTcRows + row);
                asm volatile("bar.sync %0, 256;" ::"r"(1 + w) : "memory");
                tab_head = g;
            }
            if (!WHOLE && !ok) continue;
            if (sums && warp_live && g != dg_head) {
                if (dg_head >= 0) dg.finish(lane);
                dg.start(diag_w + g * (2 * a.M + 1));
                dg_head = g;
            }
            chunks(i, ca, cb);
            const bool on = warp_live && c >= ca && c < cb;
            // the scores, and (the loads' own barrier) the queries' stats
            ok = warp_wait(&full[s], (t / kSlots) & 1, abort) && warp_wait(&s_full[w], (t >> 1) & 1, abort);
            if (!ok) {
                if (WHOLE) break;
                continue;
            }
            tc_fence_after();
            uint32_t x[32], y[32];
            if (on) {
                const float4* st = stat_s + s * (C::stat / 16) + c * (kTcChunk / 2);  // lse, delta of two queries each
                tmem_ld32_async(at_s, x);
                tmem_ld_wait(x);
                if (BIAS) {
                    // relative positions k0 - (start + ic + 31) ... k1 - 1 - (start + ic)
                    const int side = k0 - (start + ic + kTcChunk - 1) >= a.M ? 1 : k1 - 1 - (start + ic) <= -a.M ? -1 : 0;
                    const float* tab = table + (WHOLE ? g : w) * sh.floats;
                    if (side) {
                        const float bb = tab[side > 0 ? sh.floats - 1 : 0];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) fma2(x[e], x[e + 1], sc, bb);
                    } else {
                        tab += a.M + kTableExtra + j - start - ic;
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), sc, tab[-e]));
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float4 u = st[e >> 1];
                    if (BIAS) {
                        x[e] = __float_as_uint(ex2((__uint_as_float(x[e]) - u.x) * kLog2e));
                        x[e + 1] = __float_as_uint(ex2((__uint_as_float(x[e + 1]) - u.z) * kLog2e));
                    } else {
                        x[e] = __float_as_uint(ex2(fmaf(__uint_as_float(x[e]), sc, -u.x)));
                        x[e + 1] = __float_as_uint(ex2(fmaf(__uint_as_float(x[e + 1]), sc, -u.z)));
                    }
                }
                if (far) {
                    const float weight = weights[(static_cast<long long>(n) * a.Hq + hk * a.G + g) * padded_queries(a.Lq) + ic + lane];  // of query ic + lane
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * __shfl_sync(0xffffffffu, weight, e));
                }
            }
            if (!(ok = warp_wait(&e_full[w], (t >> 1) & 1, abort))) {
                if (WHOLE) break;
                continue;
            }
            tc_fence_after();
            if (on) {
                const float4* st = stat_s + s * (C::stat / 16) + c * (kTcChunk / 2);
                tmem_ld32_async(at_s + 64, y);
                tmem_ld_wait(y);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float4 u = st[e >> 1];
                    y[e] = __float_as_uint(__uint_as_float(x[e]) * (__uint_as_float(y[e]) - u.y));
                    y[e + 1] = __float_as_uint(__uint_as_float(x[e + 1]) * (__uint_as_float(y[e + 1]) - u.w));
                }
                if (ic < all_lo || ic > all_hi) {
                    const uint32_t see = low_bits(vhi - ic) & ~low_bits(vlo - ic);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(see & (1u << e))) x[e] = y[e] = 0u;
                }
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = pack2<T>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                tmem_st16(at_s, p);
                if (EXACT) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[e] = pack_low<T>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), p[e]);
                    tmem_st16(at_s + kLow, p);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = pack2<T>(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
                tmem_st16(at_s + 64, p);
                if (EXACT) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[e] = pack_low<T>(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]), p[e]);
                    tmem_st16(at_s + 64 + kLow, p);
                }
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[w]));
            if (sums && on) {  // under the products that p and d go into
                const bool above = kw - (start + ic + kTcChunk - 1) >= a.M, below = kw + 31 - (start + ic) <= -a.M;
                if (above || below) {
                    float2 sum[2] = {};
#pragma unroll
                    for (int e = 0; e < 32; e += 2) add2(sum[(e >> 1) & 1], y[e], y[e + 1]);
                    (above ? dg.above : dg.below) += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                } else {
                    dg.chunk(ic, lane, y);
                }
            }
            s += 2;
            if (s >= kSlots) s -= kSlots;
        }
        if (sums && dg_head >= 0) dg.finish(lane);
        if (ok && cnt) ok = warp_wait(&done, 0u, abort);
        tc_fence_after();
        // parity 0 stores gv, 1 gk, each chunk's warps every second 32 columns
        const bool row_here = parts > 1 || j < a.Lk;
        const uint32_t at_o = lane_base + 256 + w * 64 * NB;
        const float f = w ? a.scale : 1.f;
        const bool zero = !cnt || j >= klen;
        T* to = (w ? gk : gv) + ((static_cast<long long>(n) * a.Lk + j) * a.Hk + hk) * a.D;
        float* po = part + ((static_cast<long long>(s_part) * 2 + w) * kTcRows + row) * a.D;
        for (int d = 32 * c; d < a.D && ok; d += 64) {
            uint32_t x[32];
            if (cnt) {
                tmem_ld32_async(at_o + d, x);
                tmem_ld_wait(x);
            }
            if (!row_here) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = zero ? 0u : __float_as_uint(__uint_as_float(x[e]) * f);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                if (d + e >= a.D) continue;
                if (parts > 1) {
                    *reinterpret_cast<uint4*>(po + d + e) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                    *reinterpret_cast<uint4*>(po + d + e + 4) = make_uint4(x[e + 4], x[e + 5], x[e + 6], x[e + 7]);
                } else {
                    uint32_t u[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) u[v] = pack2<T>(__uint_as_float(x[e + 2 * v]), __uint_as_float(x[e + 2 * v + 1]));
                    *reinterpret_cast<uint4*>(to + d + e) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort) kv_gave_up<T>(a, sh, gk, gv, part, BIAS ? diag : nullptr);
    if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem));
}

// Sums the parts of tiles that were split, in order: a thread per four entries.
template <typename T>
__global__ void __launch_bounds__(256) kv_join_kernel(BandArgs a, KvShape sh, int tiles, const float* __restrict__ part,
                                                      T* __restrict__ gk, T* __restrict__ gv) {
    const int D4 = a.D / 4;
    const long long per = static_cast<long long>(tiles) * kTcRows * D4 * 2, e = blockIdx.x * 256ll + threadIdx.x;
    if (e >= per * a.N * a.Hk) return;
    const long long nh = e / per;
    long long r = e - nh * per;
    const int d = static_cast<int>(r % D4) * 4;
    r /= D4;
    const int row = static_cast<int>(r % kTcRows);
    r /= kTcRows;
    const int side = static_cast<int>(r & 1), kt = static_cast<int>(r >> 1), j = kt * kTcRows + row;
    if (j >= a.Lk) return;
    const bool sink = kt < sh.sink_tiles;
    const int parts = sink ? sh.sink_parts : sh.other_parts;
    if (parts == 1) return;
    const int first = sink ? kt * parts : sh.sink_tiles * sh.sink_parts + (kt - sh.sink_tiles) * parts;
    const float* p = part + (((nh * (sh.items() - sh.whole) + first) * 2 + side) * kTcRows + row) * a.D + d;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(p + static_cast<long long>(i) * 2 * kTcRows * a.D);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const long long n = nh / a.Hk, hk = nh - n * a.Hk;
    T* to = (side ? gk : gv) + ((n * a.Lk + j) * a.Hk + hk) * a.D + d;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack2<T>(s.x, s.y), pack2<T>(s.z, s.w));
}

// How the rows of grad_q map to its CTAs: two tiles of `tq` queries of `pack` heads each.
struct RowShape {
    int pack, tq, blocks;
};
// Whether the bias tables of all heads that share a key head fit shared memory beside the tiles.  If not,
// grad_q's tiles are of one head, and grad_kv, which goes head by head, reloads its table at each.
bool whole_tables(const BandArgs& a) {
    return !a.nb || static_cast<size_t>(a.G) * table_floats(a.M) * sizeof(float) <= kTableBytes;
}
RowShape row_shape(const BandArgs& a) {
    const int pack = whole_tables(a) ? a.G : 1, tq = kTcRows / pack;
    return {pack, tq, (a.Lq + 2 * tq - 1) / (2 * tq)};
}

KvShape kv_shape(const BandArgs& a) {
    KvShape s;
    s.floats = a.nb ? table_floats(a.M) : 0;
    s.tiles = (a.Lk + kTcRows - 1) / kTcRows;
    // the tiles a window leaves behind see about `left + right` queries, those of the sinks all that follow
    const long long reach = std::min<long long>(a.Lq, static_cast<long long>(std::min(a.left, kBandMaxLen)) + std::min(a.right, kBandMaxLen) + kTcRows);
    s.sink_tiles = a.left < kBandFar ? std::min((a.sinks + kTcRows - 1) / kTcRows, s.tiles) : 0;
    const int wide = (a.Lq + kTile - 1) / kTile, narrow = static_cast<int>((reach + kTile - 1) / kTile) + 1;
    // parts until every SM has a CTA, none shorter than four steps
    const long long ctas = static_cast<long long>(a.N) * a.Hk * s.tiles;
    const long long want = std::max<long long>(1, kBandSms / ctas);
    s.other_parts = static_cast<int>(std::min<long long>(want, std::max<long long>(1, static_cast<long long>(narrow) * a.G / 4)));
    s.sink_parts = s.other_parts;
    if (s.sink_tiles) {  // parts about as long as a window, while that keeps the parts' memory small
        const long long each = static_cast<long long>(a.N) * a.Hk * s.sink_tiles, most = (4 * kBandSms + each - 1) / each;
        s.sink_parts = static_cast<int>(std::max<long long>(s.other_parts, std::min<long long>(static_cast<long long>(s.other_parts) * ((wide + narrow - 1) / narrow), most)));
    }
    s.whole = s.other_parts > 1 ? 0 : s.items() - s.sink_tiles * s.sink_parts;
    return s;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }
size_t stats_bytes(const BandArgs& a) { return up256(static_cast<size_t>(a.N) * a.Hq * padded_queries(a.Lq) * sizeof(float2)); }
size_t far_bytes(const BandArgs& a) {
    const RowShape r = row_shape(a);
    return up256(static_cast<size_t>(a.N) * (a.Hq / r.pack) * r.blocks * sizeof(int));
}
size_t weights_bytes(const BandArgs& a) { return up256(static_cast<size_t>(a.N) * a.Hq * padded_queries(a.Lq) * sizeof(float)); }
size_t part_bytes(const BandArgs& a, const KvShape& s) {
    return s.split() ? up256(static_cast<size_t>(a.N) * a.Hk * (s.items() - s.whole) * 2 * kTcRows * a.D * sizeof(float)) : 0;
}
size_t diag_bytes(const BandArgs& a, const KvShape& s) {
    return a.nb ? up256(static_cast<size_t>(a.N) * a.Hq * s.items() * kDiagWarps * (2 * a.M + 1) * sizeof(float)) : 0;
}
size_t sums_bytes(const BandArgs& a) { return a.nb ? up256(band_sum_bytes(a)) : 0; }

template <typename T, int NB, bool BIAS, bool EXACT>
cudaError_t launch(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq, void* gk, void* gv, void* gbias,
                   void* ws, cudaStream_t stream) {
    char* at = static_cast<char*>(ws);
    const KvShape kv = kv_shape(a);
    float2* stats = reinterpret_cast<float2*>(at);
    float* weights = reinterpret_cast<float*>(at += stats_bytes(a));
    int* far_blocks = reinterpret_cast<int*>(at += weights_bytes(a));
    float* part = reinterpret_cast<float*>(at += far_bytes(a));
    float* diag = BIAS && gbias ? reinterpret_cast<float*>(at += part_bytes(a, kv)) : nullptr;
    float* sums = diag ? reinterpret_cast<float*>(at += diag_bytes(a, kv)) : nullptr;
    const auto [pack, tq, blocks] = row_shape(a);
    const bool whole = !BIAS || whole_tables(a);
    const long long dense = static_cast<long long>(a.Hq) * a.D;
    const size_t smem_q = QCfg<NB, BIAS>::smem + (BIAS ? static_cast<size_t>(pack) * kv.floats * sizeof(float) : 0),
                 smem_kv = KvCfg<NB, BIAS>::smem + (BIAS ? static_cast<size_t>(whole ? a.G : 2) * kv.floats * sizeof(float) : 0);
    cudaError_t e = allow_smem<grad_q_kernel<T, NB, BIAS, EXACT>>();
    if (e == cudaSuccess) e = whole ? allow_smem<grad_kv_kernel<T, NB, BIAS, EXACT, true>>() : allow_smem<grad_kv_kernel<T, NB, BIAS, EXACT, !BIAS>>();
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mg, mk, mv, mq1, mg1, mk1, mv1;
    if (!make_map(&mq, a.dtype, a.q, a.N, a.Lq, a.Hq, a.D, a.q_batch, a.q_row, pack, tq) ||
        !make_map(&mg, a.dtype, gout, a.N, a.Lq, a.Hq, a.D, dense * a.Lq, dense, pack, tq) ||
        !make_map(&mk, a.dtype, a.k, a.N, a.Lk, a.Hk, a.D, a.k_batch, a.k_row, 1, kTile) ||
        !make_map(&mv, a.dtype, a.v, a.N, a.Lk, a.Hk, a.D, a.v_batch, a.v_row, 1, kTile) ||
        !make_map(&mq1, a.dtype, a.q, a.N, a.Lq, a.Hq, a.D, a.q_batch, a.q_row, 1, kTile) ||
        !make_map(&mg1, a.dtype, gout, a.N, a.Lq, a.Hq, a.D, dense * a.Lq, dense, 1, kTile) ||
        !make_map(&mk1, a.dtype, a.k, a.N, a.Lk, a.Hk, a.D, a.k_batch, a.k_row, 1, kTcRows) ||
        !make_map(&mv1, a.dtype, a.v, a.N, a.Lk, a.Hk, a.D, a.v_batch, a.v_row, 1, kTcRows))
        return cudaErrorInvalidValue;
    int lanes = 1;
    while (lanes * 8 < a.D) lanes *= 2;
    const int each = 4 * 256 / lanes;
    const long long row_blocks = static_cast<long long>(a.N) * a.Hq * ((padded_queries(a.Lq) + each - 1) / each);
    stats_kernel<T><<<static_cast<unsigned>(row_blocks), 256, 0, stream>>>(a, lanes, static_cast<const T*>(out), lse,
                                                                                      static_cast<const T*>(gout), stats, weights);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    grad_q_kernel<T, NB, BIAS, EXACT><<<static_cast<unsigned>(static_cast<long long>(a.N) * (a.Hq / pack) * blocks), QCfg<NB, BIAS>::threads, smem_q, stream>>>(
        mq, mg, mk, mv, a, pack, tq, blocks, kv.floats, stats, weights, far_blocks, static_cast<T*>(gq));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const auto kv_kernel = whole ? grad_kv_kernel<T, NB, BIAS, EXACT, true> : grad_kv_kernel<T, NB, BIAS, EXACT, !BIAS>;
    kv_kernel<<<static_cast<unsigned>(static_cast<long long>(a.N) * a.Hk * kv.items()), KvCfg<NB, BIAS>::threads, smem_kv, stream>>>(
        mq1, mg1, mk1, mv1, a, kv, stats, weights, far_blocks, blocks * (a.G / pack), static_cast<T*>(gk), static_cast<T*>(gv), part, diag);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (kv.split()) {
        const int tiles = kv.other_parts > 1 ? kv.tiles : kv.sink_tiles;
        const long long n4 = static_cast<long long>(a.N) * a.Hk * tiles * kTcRows * (a.D / 4) * 2;
        kv_join_kernel<T><<<static_cast<unsigned>((n4 + 255) / 256), 256, 0, stream>>>(a, kv, tiles, part, static_cast<T*>(gk), static_cast<T*>(gv));
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return diag ? launch_band_bias_sum(a, kv.items(), kDiagWarps, diag, sums, gbias, stream) : cudaSuccess;
}

}  // namespace

size_t band_bwd_tc_workspace(const BandArgs& a, bool want_bias) {
    const KvShape kv = kv_shape(a);
    return stats_bytes(a) + weights_bytes(a) + far_bytes(a) + part_bytes(a, kv) + (want_bias ? diag_bytes(a, kv) + sums_bytes(a) : 0);
}

cudaError_t launch_band_bwd_tc(const BandArgs& a, const void* out, const float* lse, const void* gout, void* gq, void* gk, void* gv,
                               void* gbias, void* ws, cudaStream_t stream) {
#define DCN4_BAND_BWD(T, NB, BIAS)                                                                          \
    (band_most_keys(a) <= kBandExactKeys ? launch<T, NB, BIAS, true>(a, out, lse, gout, gq, gk, gv, gbias, ws, stream) \
                                     : launch<T, NB, BIAS, false>(a, out, lse, gout, gq, gk, gv, gbias, ws, stream))
#define DCN4_BAND_BWD_T(T)                                                                    \
    (a.D > 64 ? (a.nb ? DCN4_BAND_BWD(T, 2, true) : DCN4_BAND_BWD(T, 2, false))               \
              : (a.nb ? DCN4_BAND_BWD(T, 1, true) : DCN4_BAND_BWD(T, 1, false)))
    return a.dtype == 1 ? DCN4_BAND_BWD_T(__half) : DCN4_BAND_BWD_T(__nv_bfloat16);
#undef DCN4_BAND_BWD_T
#undef DCN4_BAND_BWD
}

cudaError_t band_bwd_status(unsigned* status, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_band_bwd_status, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_band_bwd_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace dcn4
