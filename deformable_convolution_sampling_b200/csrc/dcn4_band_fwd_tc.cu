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
// share a key head) and streams tiles of keys past both, or, where a head has
// no more than one tile of rows, lets its two halves take the key tiles in turn.
// Warps 0-3 and 4-7 each own a tile's softmax (thread = row = TMEM lane), warp 8
// loads tiles with TMA, the warps from 9 on issue the MMAs:
//     S = Q K^T  (both operands in shared memory, into tensor memory)
//     O += P V   (P written over S in tensor memory as 16-bit pairs)
// so that one tile's exponentials run under the other's products.  Of a key tile
// only the 32-column chunks that some row may see are computed; only chunks on the
// band's edge are masked element by element.
//
// Bound by MMAs of N = 64 from shared memory (49 cycles, not 32: its bandwidth) and by
// exponentials in equal parts for heads of 128; for heads of 32 with a bias by what a
// pair costs beside its exponential (a shared read of its bias near the diagonal, mask,
// maximum) on eight softmax warps a CTA: 52 % of the issue slots, 9 % of the tensor pipe.
// Tiles of 128 keys would run the MMAs at their full rate, but leave tensor memory room
// for one tile's scores a half: 203 us against 145 at 8192 causal tokens with a window of
// 2048 and 16 heads of 128 on 4, before an issuing warp a half and waits that end on a
// vote; not measured since.  That call now: 147 us (818 TFLOP/s); 8 maps of 64 x 64, eight
// rows of pixels and a bias, 8 heads of 32: 123 us.
#include "dcn4_band_tc.cuh"

namespace dcn4 {
namespace {

using namespace tc;

constexpr int kProducer = 8, kMma = 9;
constexpr float kRescale = 8.f;
constexpr int kTableExtra = 160;      // the bias table reaches past M by a tile's rows and a chunk: no clamp in a chunk that touches [-M, M]

// Tiles of 64 keys.  Heads up to 128: the scores of two tiles a half in tensor
// memory, so that the product for tile t + 1 runs under the exponentials of tile t.
// Heads of up to 64: one, in 256 columns of tensor memory, and two CTAs an SM.
constexpr int kKeys = 64, kChunks = kKeys / kTcChunk;
constexpr int kKeyBlock = kKeys * 128;                   // bytes of 64 columns of a key tile
template <int NB>
struct Cfg {
    static constexpr int ahead = NB == 1 ? 1 : 2;        // tiles whose scores are held
    static constexpr int mma = NB == 1 ? 1 : 2;          // warps that issue: one for both halves, or one for each
    static constexpr int threads = (kMma + mma) * 32;
    static constexpr int slots = 4;                      // ring of V of a tile with K of the tile `ahead` on
    static constexpr int scores = ahead * kKeys;         // columns of a half's scores
    static constexpr int tmem = NB == 1 ? 256 : 512;
    static constexpr int ctas = NB == 1 ? 2 : 1;
    static constexpr int table_bytes = NB == 1 ? 12 << 10 : 28 << 10;
};

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
    int lo = max(b.lo, j0), hi = min(b.hi, j0 + kKeys);
    const int sink = min(b.sink, j0 + kKeys);
    if (sink > j0) {
        if (lo >= hi) hi = sink;
        lo = j0;
    }
    ca = (lo - j0) >> 5;
    cb = (hi - j0 + kTcChunk - 1) >> 5;
    return b.any && lo < hi;
}

// After a wait that gave up: the block's results are NaN, and the status word says so.  (A call, with nothing of the
// kernel's own, so that its registers are those of the way without it: as part of the kernel it cost 2 %.)
template <typename T>
__device__ __noinline__ void fwd_gave_up(BandArgs a, FwdShape sh, T* out, float* lse, BandPart part) {
    if (threadIdx.x == 0) atomicOr(&g_band_status, 1u);
    int b = blockIdx.x;
    const int sp = b % sh.splits;
    b /= sh.splits;
    const int blk = sh.blocks - 1 - b % sh.blocks;
    b /= sh.blocks;
    const int groups = a.Hq / sh.pack, n = b / groups, h0 = (b - n * groups) * sh.pack, queries = (sh.alt ? 1 : 2) * sh.tq;
    const int i0 = blk * queries, rows = max(min(i0 + queries, a.Lq) - i0, 0) * sh.pack;
    for (int r = threadIdx.x; r < rows; r += blockDim.x) {
        const int i = i0 + r / sh.pack, h = h0 + r % sh.pack;
        const long long at = (static_cast<long long>(n) * a.Hq + h) * a.Lq + i;
        if (sh.splits > 1) {
            fill_nan(&part.ml[at * sh.splits + sp].y, 1);
        } else {
            fill_nan(lse + at, 1);
            fill_nan(out + ((static_cast<long long>(n) * a.Lq + i) * a.Hq + h) * a.D, a.D);
        }
    }
}

// EXACT: p as two numbers (kBandExactKeys)
template <typename T, int NB, bool BIAS, bool EXACT>
__global__ void __launch_bounds__(Cfg<NB>::threads, Cfg<NB>::ctas)
    fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, BandArgs a, FwdShape sh, T* __restrict__ out,
               float* __restrict__ lse, BandPart part) {
    using C = Cfg<NB>;
    constexpr int kSlots = C::slots, kAhead = C::ahead;
    extern __shared__ __align__(1024) unsigned char band_smem[];
    __shared__ __align__(8) uint64_t full[kSlots], empty[kSlots], raw, q_full, s_full[2][2], p_full[2][2], o_done[2][2], drained[2];
    __shared__ uint32_t taddr_s;
    __shared__ int s_abort;
    __shared__ float2 s_ml[kTcRows];
    const int tid = threadIdx.x, warp = static_cast<int>(uniform(tid >> 5)), lane = tid & 31;
    const uint32_t base = (smem_u32(band_smem) + 1023u) & ~1023u;
    const uint32_t qs = base, ring = base + (sh.alt ? 1 : 2) * NB * kTcBlock;
    float* table = reinterpret_cast<float*>(band_smem + (ring - smem_u32(band_smem)) + kSlots * 2 * NB * kKeyBlock);

    int b = blockIdx.x;
    const int sp = b % sh.splits;
    b /= sh.splits;
    const int blk = sh.blocks - 1 - b % sh.blocks;  // the longest rows of a causal band first
    b /= sh.blocks;
    const int groups = a.Hq / sh.pack, n = b / groups, grp = b - n * groups, h0 = grp * sh.pack, hk = h0 / a.G;
    const int klen = static_cast<int>(uniform(band_klen(a, n))), qlen = static_cast<int>(uniform(band_qlen(a, n))),
              start = static_cast<int>(uniform(band_start(a, n)));
    const int tiles = sh.alt ? 1 : 2;
    const int i0 = blk * tiles * sh.tq, i1 = min(i0 + tiles * sh.tq, qlen) - 1;

    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), C::mma);
        }
        mbar_init(smem_u32(&drained[0]), 1);
        mbar_init(smem_u32(&drained[1]), 1);
        mbar_init(smem_u32(&raw), 1);
        mbar_init(smem_u32(&q_full), 1);
        for (int w = 0; w < 4; ++w) {
            mbar_init(smem_u32(&s_full[w >> 1][w & 1]), 1);
            mbar_init(smem_u32(&p_full[w >> 1][w & 1]), 4);
            mbar_init(smem_u32(&o_done[w >> 1][w & 1]), 1);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kProducer && elect_one()) {
        prefetch_map(&map_q);
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    if (warp == kMma) {  // S and O of both halves
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&taddr_s)), "r"(C::tmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (BIAS) {  // the bias of every head of the tile by relative position
        for (int e = tid; e < sh.pack * sh.table; e += C::threads) {
            const int g = e / sh.table, rel = e - g * sh.table - a.M - kTableExtra;
            const int bk = __ldg(a.buckets + max(-a.M, min(rel, a.M)) + a.M);
            table[e] = static_cast<unsigned>(bk) < static_cast<unsigned>(a.nb)
                           ? to_f32(static_cast<const T*>(a.bias)[static_cast<long long>(bk) * a.Hq + h0 + g]) : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(taddr_s);
    volatile int* abort = &s_abort;

    int t0 = 0, t1 = 0;
    BandTiles bt{0, 0, 0};
    if (i0 <= i1) {
        bt = band_tiles(a, start + i0, start + i1, klen, kKeys);
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
        return chunks_of(w ? rb1 : rb0, bt.tile(t) * kKeys, ca, cb);
    };

    if (warp == kProducer) {
        if (t0 < t1 && elect_one()) {
            const int bytes = sh.pack * sh.tq * 128;
            mbar_expect_tx(smem_u32(&q_full), tiles * NB * bytes);
            for (int w = 0; w < tiles; ++w)
                for (int c = 0; c < NB; ++c)
                    tma_load_rows(qs + (w * NB + c) * kTcBlock, &map_q, c * 64, h0, i0 + w * sh.tq, n, smem_u32(&q_full));
        }
        // stage i: K of tile i and V of tile i - kAhead
        int raws = 0;
        const int cnt = t1 - t0;
        for (int i = 0; cnt && i < cnt + kAhead; ++i) {
            const int s = i % kSlots;
            if (!warp_wait(&empty[s], ((i / kSlots) & 1) ^ 1u, abort)) break;
            const uint32_t at_k = ring + s * 2 * NB * kKeyBlock, at_v = at_k + NB * kKeyBlock;
            const bool with_k = i < cnt, with_v = i >= kAhead;
            const int jv = with_v ? bt.tile(t0 + i - kAhead) * kKeys : 0;
            // values past the sequence but inside the tensor meet probabilities of 0: clear them (scores are masked)
            const bool clear = with_v && jv + kKeys > klen && klen < a.Lk;
            if (elect_one()) {
                const uint32_t bar = smem_u32(clear ? &raw : &full[s]);
                mbar_expect_tx(bar, (with_k + with_v) * NB * kKeyBlock);
                const int jk = with_k ? bt.tile(t0 + i) * kKeys : 0;
                for (int c = 0; c < NB; ++c) {
                    if (with_k) tma_load_rows(at_k + c * kKeyBlock, &map_k, c * 64, hk, jk, n, bar);
                    if (with_v) tma_load_rows(at_v + c * kKeyBlock, &map_v, c * 64, hk, jv, n, bar);
                }
            }
            if (clear) {
                if (!warp_wait(&raw, raws++ & 1, abort)) break;
                zero_rows<NB>(at_v, kKeyBlock, max(klen - jv, 0), kKeys, lane);
                if (elect_one()) mbar_arrive(smem_u32(&full[s]));
            }
        }
    } else if (warp >= kMma) {
        if (t0 < t1) {
            const int steps = (a.D + 15) / 16;
            // a negative scale turns the products' sign, so that the largest score is the largest product
            const uint32_t id_s = umma_idesc<T>(kTcRows, 0, 0, 0) | (a.scale < 0.f ? kNegateA : 0u),
                           id_o = umma_idesc<T>(kTcRows, steps * 16, 0, 1);
            const uint64_t q_desc = umma_desc_sw128(qs, 16, 1024), k_desc = umma_desc_sw128(ring, 16, 1024),
                           v_desc = umma_desc_sw128(ring + NB * kKeyBlock, kKeyBlock, 1024);
            const int w_lo = C::mma == 2 ? warp - kMma : 0, w_hi = C::mma == 2 ? w_lo + 1 : 2;
            bool ok = warp_wait(&q_full, 0u, abort);
            uint32_t counts = 0;  // scores (bits 0-1) and sums (2-3) issued by each half, mod 2; whether it has an O (4-5)
            int now0 = -1, now1 = -1, ahead0 = -1, ahead1 = -1;  // chunks of each half's tile, ca | cb << 8 (-1: none), and of the next with kAhead 2
            uint32_t phases = 0;  // of p_full[w][buf], bit 2 w + buf
            auto span_of = [&](int w, int t) {
                int ca, cb;
                return active(w, t, ca, cb) ? ca | cb << 8 : -1;
            };
            auto scores = [&](int w, int s, int span) {
                const int buf = kAhead == 2 ? (counts >> w) & 1 : 0, ca = span & 255, cb = span >> 8;
                counts ^= 1u << w;
                if (elect_one()) {
                    issue_rows<NB>(tmem + w * C::scores + buf * kKeys + ca * kTcChunk, step_desc(q_desc, sh.alt ? 0 : w * NB * kTcBlock), kTcBlock,
                                   step_desc(k_desc, s * 2 * NB * kKeyBlock + ca * kTcChunk * 128), kKeyBlock,
                                   id_s | (static_cast<uint32_t>((cb - ca) * (kTcChunk / 8)) << 17), steps);
                    umma_commit(smem_u32(&s_full[w][buf]));
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int i = 0; i < kAhead && ok; ++i) {
                if (t0 + i >= t1) break;
                if (!(ok = warp_wait(&full[i], 0u, abort))) break;
                tc_fence_after();
#pragma unroll 1
                for (int w = w_lo; w < w_hi; ++w) {
                    const int span = span_of(w, t0 + i);
                    if (i == 0) (w ? now1 : now0) = span; else (w ? ahead1 : ahead0) = span;
                    if (span >= 0) scores(w, i, span);
                }
                if (elect_one()) umma_commit(smem_u32(&empty[i]));
                __syncwarp();
            }
            int s = kAhead;
            uint32_t ph = 0;
#pragma unroll 1
            for (int t = t0; t < t1 && ok; ++t) {
                const int next0 = w_lo == 0 ? span_of(0, t + kAhead) : -1, next1 = w_hi == 2 ? span_of(1, t + kAhead) : -1;
                if (!(ok = warp_wait(&full[s], ph, abort))) break;
                tc_fence_after();
                // first the halves that rest on this tile: they start on the next one at once
#pragma unroll 1
                for (int u = 2 * w_lo; u < 2 * w_hi; ++u) {
                    const int w = C::mma == 2 ? w_lo : u & 1, now = w ? now1 : now0, next = w ? next1 : next0;
                    if ((C::mma == 2 ? !(u & 1) : u < 2) != (now < 0)) continue;
                    if (now >= 0) {
                        const int buf = kAhead == 2 ? (counts >> (2 + w)) & 1 : 0;
                        ok = warp_wait(&p_full[w][buf], (phases >> (2 * w + buf)) & 1u, abort);
                        if (!ok) break;
                        tc_fence_after();
                        phases ^= 1u << (2 * w + buf);
                        if (elect_one()) {
                            issue_sum<kKeys / 16>(tmem + 2 * C::scores + w * 64 * NB, tmem + w * C::scores + buf * kKeys,
                                                  step_desc(v_desc, s * 2 * NB * kKeyBlock), id_o, (now & 255) * 2, (now >> 8) * 2,
                                                  (counts >> (4 + w)) & 1);
                            if (EXACT)
                                issue_sum<kKeys / 16>(tmem + 2 * C::scores + w * 64 * NB, tmem + w * C::scores + buf * kKeys + kLow,
                                                      step_desc(v_desc, s * 2 * NB * kKeyBlock), id_o, (now & 255) * 2, (now >> 8) * 2, true);
                            umma_commit(smem_u32(&o_done[w][buf]));
                        }
                        __syncwarp();
                        counts ^= 4u << w;
                        counts |= 16u << w;
                    }
                    if (next >= 0) scores(w, s, next);  // after the product that reads P, whose place its S takes
                }
                if (!ok) break;
                if (elect_one()) umma_commit(smem_u32(&empty[s]));
                __syncwarp();
                s = s + 1 == kSlots ? 0 : s + 1;
                ph ^= s == 0;
                if (kAhead == 2) {
                    now0 = ahead0;
                    now1 = ahead1;
                    ahead0 = next0;
                    ahead1 = next1;
                } else {
                    now0 = next0;
                    now1 = next1;
                }
            }
            if (!ok && lane == 0) {  // the MMAs already issued must end before the memory goes
                umma_commit(smem_u32(&drained[warp - kMma]));
                int never = 0;
                mbar_wait_or(smem_u32(&drained[warp - kMma]), 0u, &never);
            }
        }
        __syncwarp();
    } else if (warp < kProducer) {
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_first = lane_base + w * C::scores, o_at = lane_base + 2 * C::scores + w * 64 * NB;
        const int ql = row / sh.pack, g = row - ql * sh.pack, i = i0 + (sh.alt ? 0 : w) * sh.tq + ql;
        const bool live = ql < sh.tq && i < qlen;
        const bool warp_live = __any_sync(0xffffffffu, live);
        const RowBand& rb = w ? rb1 : rb0;
        const int pos = start + i;
        const int jlo = max(0, pos - a.left), jhi = min(klen, pos + a.right + 1), jsink = min(a.sinks, jhi);
        // keys that every row of the tile sees; relative positions at which a chunk has one bias
        const int all_lo = rb.phi - a.left, all_hi = min(klen, rb.plo + a.right + 1) - kTcChunk;
        float rm = -INFINITY, rl = 0.f;  // reference (log2 units without a bias, natural with one) and sum
        // a scale of 0 is held at 1e-38, so that 0 times a mask's infinity does not arise (a normal number, also times
        // log2 e; products below 1e31 still vanish next to any score)
        const float scale = a.scale == 0.f ? 1e-38f : fabsf(a.scale);
        const float sc = BIAS ? scale : scale * kLog2e;
        constexpr float unit = BIAS ? kLog2e : 1.f;  // of the reference, to log2
        const float* tab = table + g * sh.table + a.M + kTableExtra - pos;
        int nw = 0, ca, cb;
        bool ok = true;
        for (int t = t0; t < t1; ++t) {
            if (!active(w, t, ca, cb)) continue;
            const int j0 = bt.tile(t) * kKeys, buf = nw & (kAhead - 1);
            const uint32_t s_at = s_first + buf * kKeys;
            ok = warp_wait(&s_full[w][buf], (nw / kAhead) & 1, abort);
            if (!ok) break;
            tc_fence_after();
            if (warp_live) {
                float mx[2] = {-INFINITY, -INFINITY};
                uint32_t x[kChunks][32];
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (c >= ca && c < cb) tmem_ld32_async(s_at + c * kTcChunk, x[c]);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (c >= ca && c < cb) {
                        const int j = j0 + c * kTcChunk;
                        tmem_ld_wait(x[c]);
                        if (BIAS) {  // natural scores with their bias: each pair's own, or that of all pairs beyond M
                            const int side = j - rb.phi >= a.M ? sh.table - 1 : 0;
                            if (side || j + kTcChunk - 1 - rb.plo <= -a.M) {
                                const float bb = table[g * sh.table + side];
#pragma unroll
                                for (int e = 0; e < 32; e += 2) fma2(x[c][e], x[c][e + 1], sc, bb);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[c][e] = __float_as_uint(fmaf(__uint_as_float(x[c][e]), sc, tab[j + e]));
                            }
                        }
                        if (j < all_lo || j > all_hi) {
                            const uint32_t see = (low_bits(jhi - j) & ~low_bits(jlo - j)) | low_bits(jsink - j);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see & (1u << e))) x[c][e] = __float_as_uint(-INFINITY);
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
                    }
                float top = fmaxf(mx[0], mx[1]);
                if (!BIAS) top *= sc;
                if (nw == 0) {
                    rm = top;
                } else if (__any_sync(0xffffffffu, live && (top - rm) * unit > kRescale)) {
                    // a maximum outgrew its reference (or a row sees its first key): move the references
                    const float to = fmaxf(top, rm);
                    const float f = to == -INFINITY ? 1.f : ex2((rm - to) * unit);
                    rm = to;
                    rl *= f;
                    ok = warp_wait(&o_done[w][(nw - 1) & (kAhead - 1)], ((nw - 1) / kAhead) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    for (int d = 0; d < a.D; d += 16) {
                        uint32_t o[16];
                        tmem_ld16(o_at + d, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(o_at + d, o);
                    }
                }
                const float ref = rm == -INFINITY ? 0.f : rm;
                float2 sum[2] = {};
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    if (c < ca || c >= cb) continue;
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        uint32_t &lo = x[c][e], &hi = x[c][e + 1];
                        if (BIAS) {  // the difference first: scores may be of the type's lowest value
                            sub_mul2(lo, hi, ref, kLog2e);
                        } else {
                            fma2(lo, hi, sc, -ref);
                        }
                        lo = __float_as_uint(ex2(__uint_as_float(lo)));
                        hi = __float_as_uint(ex2(__uint_as_float(hi)));
                        add2(sum[(e >> 1) & 1], lo, hi);
                        p[e >> 1] = pack2<T>(__uint_as_float(lo), __uint_as_float(hi));
                    }
                    tmem_st16(s_at + c * kTcChunk, p);  // the scores are in registers: P takes their place
                    if (EXACT) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = pack_low<T>(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1]), p[e]);
                        tmem_st16(s_at + c * kTcChunk + kLow, p);
                    }
                }
                rl += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st_wait();
            }
            ++nw;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[w][buf]));
        }
        if (ok && nw > 0) ok = warp_wait(&o_done[w][(nw - 1) & (kAhead - 1)], ((nw - 1) / kAhead) & 1, abort);
        tc_fence_after();
        if (sh.alt) {
            // the second half's rows are the first's: join them (its O is in the same lanes)
            if (w == 1) s_ml[row] = make_float2(rm, nw > 0 && warp_live ? rl : 0.f);
            tc_fence_before();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            tc_fence_after();
        }
        const bool rows_here = ql < sh.tq && i < a.Lq;
        if (ok && !(sh.alt && w == 1) && __any_sync(0xffffffffu, rows_here)) {
            // (a sum is 0 where a row sees nothing, and NaN, which must stay, where it sees one)
            float f0 = 1.f, f1 = 0.f, m = rm, l = live ? rl : 0.f;
            bool first = nw > 0, second = false;
            if (sh.alt) {
                const float2 other = s_ml[row];
                const float l1 = live ? other.y : 0.f;
                m = fmaxf(rm, l1 != 0.f ? other.x : -INFINITY);
                const float ref = m == -INFINITY ? 0.f : m;
                f0 = l != 0.f ? ex2((rm - ref) * unit) : 0.f;
                f1 = l1 != 0.f ? ex2((other.x - ref) * unit) : 0.f;
                l = l * f0 + l1 * f1;
                second = t1 - t0 > 1 && __any_sync(0xffffffffu, l1 != 0.f);
            }
            const long long at = (static_cast<long long>(n) * a.Hq + h0 + g) * a.Lq + i;
            const bool split = sh.splits > 1;
            const float inv = l != 0.f ? (split ? 1.f : 1.f / l) : 0.f;
            f0 = l != 0.f ? f0 * inv : 0.f;
            f1 *= inv;
            if (rows_here) {
                if (split)
                    part.ml[at * sh.splits + sp] = make_float2(l != 0.f ? m : -INFINITY, l);
                else
                    lse[at] = l != 0.f ? (BIAS ? m : m * kLn2) + logf(l) : -INFINITY;
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
    if (*abort) fwd_gave_up<T>(a, sh, out, lse, part);
    if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::tmem));
}

FwdShape shape_of(const BandArgs& a) {
    FwdShape s;
    const int table_bytes = a.D > 64 ? Cfg<2>::table_bytes : Cfg<1>::table_bytes;
    s.table = a.nb ? table_floats(a.M) : 0;
    s.pack = a.G;
    if (s.pack * s.table * static_cast<int>(sizeof(float)) > table_bytes) s.pack = 1;
    s.tq = kTcRows / s.pack;
    s.alt = a.Lq <= s.tq;
    s.blocks = s.alt ? 1 : (a.Lq + 2 * s.tq - 1) / (2 * s.tq);
    const long long ctas = static_cast<long long>(a.N) * (a.Hq / s.pack) * s.blocks;
    s.splits = band_splits(a, ctas, std::min(a.Lq, 2 * s.tq), kKeys, a.D > 64 ? Cfg<2>::ctas : Cfg<1>::ctas);
    return s;
}

template <typename T, int NB, bool BIAS, bool EXACT>
cudaError_t launch(const BandArgs& a, const FwdShape& s, void* out, float* lse, void* ws, cudaStream_t stream) {
    using C = Cfg<NB>;
    const size_t smem = 1024 + static_cast<size_t>(s.alt ? 1 : 2) * NB * kTcBlock + static_cast<size_t>(C::slots) * 2 * NB * kKeyBlock +
                        s.pack * s.table * sizeof(float);
    cudaError_t e = allow_smem<fwd_kernel<T, NB, BIAS, EXACT>>();
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, a.dtype, a.q, a.N, a.Lq, a.Hq, a.D, a.q_batch, a.q_row, s.pack, s.tq) ||
        !make_map(&mk, a.dtype, a.k, a.N, a.Lk, a.Hk, a.D, a.k_batch, a.k_row, 1, kKeys) ||
        !make_map(&mv, a.dtype, a.v, a.N, a.Lk, a.Hk, a.D, a.v_batch, a.v_row, 1, kKeys))
        return cudaErrorInvalidValue;
    const BandPart part = band_part(a, s.splits, ws);
    const long long ctas = static_cast<long long>(a.N) * (a.Hq / s.pack) * s.blocks * s.splits;
    fwd_kernel<T, NB, BIAS, EXACT><<<static_cast<unsigned>(ctas), C::threads, smem, stream>>>(mq, mk, mv, a, s, static_cast<T*>(out), lse, part);
    e = cudaGetLastError();
    if (e != cudaSuccess || s.splits == 1) return e;
    return launch_band_join(a, s.splits, part, BIAS ? 1.f : kLn2, out, lse, stream);
}

template <typename T, int NB>
cudaError_t launch_heads(const BandArgs& a, const FwdShape& s, void* out, float* lse, void* ws, cudaStream_t stream) {
    if (band_most_keys(a) <= kBandExactKeys)
        return a.nb ? launch<T, NB, true, true>(a, s, out, lse, ws, stream) : launch<T, NB, false, true>(a, s, out, lse, ws, stream);
    return a.nb ? launch<T, NB, true, false>(a, s, out, lse, ws, stream) : launch<T, NB, false, false>(a, s, out, lse, ws, stream);
}

template <typename T>
cudaError_t launch_typed(const BandArgs& a, void* out, float* lse, void* ws, cudaStream_t stream) {
    const FwdShape s = shape_of(a);
    return a.D > 64 ? launch_heads<T, 2>(a, s, out, lse, ws, stream) : launch_heads<T, 1>(a, s, out, lse, ws, stream);
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
