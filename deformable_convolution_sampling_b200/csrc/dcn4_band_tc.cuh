// dcn4_band_tc.cuh — what the band attention's tensor-core kernels share: operand
// tiles of 128 rows in the 128-byte swizzled layout, products whose first operand
// is in tensor memory, and tensor-memory loads and stores by a thread per row.
//
// Operand tile: rows (queries or keys) of D entries in blocks of 64 columns; row r
// of a block is 128 bytes at r * 128, its 16-byte pieces permuted by r mod 8 (what
// TMA's 128-byte swizzle writes).  As a K-major operand (contraction over D) a step
// of 16 entries moves 32 bytes, as an M/N-major one (contraction over the rows) a
// step of 16 rows moves 2048 bytes and the blocks are one block's bytes apart.
// Entries past D and rows past the tensor arrive as zeros; rows between a
// sequence's own length and the tensor's end may hold anything, and 0 times an
// infinity is not 0, so the one tile they can share is cleared there after it lands.
#pragma once

#include <type_traits>

#include "dcn4_band_parts.cuh"
#include "dcn4_common.cuh"
#include "dcn4_tcgen05.cuh"

namespace dcn4 {
namespace tc {

constexpr int kTcRows = 128;                 // rows of a tile: the MMA's M, TMEM's lanes
constexpr int kTcBlock = kTcRows * 128;      // bytes of 64 columns of a tile of 128 rows
constexpr int kTcChunk = 32;                 // columns of scores handled at a time
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A in tensor memory (16-bit pairs, 8 columns a K step of 16), B in shared memory.
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, bool accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accum ? 1 : 0));
}

// The 32 columns of this thread's lane, not waited for.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Waits for the loads above; the registers pass through so that no use moves before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t u;
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        memcpy(&u, &h, 4);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        memcpy(&u, &h, 4);
    }
    return u;
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A box of rows of an operand's tensor map (make_map): 64 columns from `col`, heads
// from `head`, tokens from `row` of image n.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int col, int head, int row, int n, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(row), "r"(n), "r"(mbar)
        : "memory");
}

// One warp writes zeros to rows [from, to) of a tile whose loads have landed.
template <int NB>
__device__ __forceinline__ void zero_rows(uint32_t tile, int block, int from, int to, int lane) {
    for (int e = from * 8 + lane; e < to * 8; e += 32)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * block + e * 16), "r"(0) : "memory");
    fence_async_smem();
    __syncwarp();
}

// A bounded wait by a whole warp: all of its lanes go on, or none.  The loop ends
// on a vote, so the warp never diverges (one lane polling for the rest took 300
// cycles on a phase long complete, this 90).
__device__ __forceinline__ bool warp_wait(uint64_t* mbar, uint32_t parity, volatile int* abort) {
    const uint32_t at = smem_u32(mbar);
    for (int i = 0; i < kTWaitSpins; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred P1;\n\tmbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
            "selp.b32 %0, 1, 0, P1;\n\t}"
            : "=r"(done)
            : "r"(at), "r"(parity)
            : "memory");
        if (__all_sync(0xffffffffu, done)) return true;
        if ((i & 63) == 63 && __any_sync(0xffffffffu, *abort)) return false;
    }
    *abort = 1;
    return false;
}

// What a block whose wait gave up leaves of a row (its copies have long landed: a wait's limit is far longer than
// they take, and without the wait's progress the ring holds back further ones).
template <typename T>
__device__ __forceinline__ void fill_nan(T* row, int n) {
    for (int d = 0; d < n; ++d) row[d] = from_f32<T>(__int_as_float(0x7fffffff));
}

// x * m + c of two values at once.
__device__ __forceinline__ void fma2(uint32_t& x, uint32_t& y, float m, float c) {
    asm("{\n\t.reg .b64 v, w, z;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 v, v, w, z;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+r"(x), "+r"(y)
        : "f"(m), "f"(c));
}
// (x - c) * m of two values at once.
__device__ __forceinline__ void sub_mul2(uint32_t& x, uint32_t& y, float c, float m) {
    asm("{\n\t.reg .b64 v, w, z;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "add.rn.f32x2 v, v, w;\n\tmul.rn.f32x2 v, v, z;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+r"(x), "+r"(y)
        : "f"(-c), "f"(m));
}
__device__ __forceinline__ void add2(float2& s, uint32_t x, uint32_t y) {
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tadd.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(s.x), "+f"(s.y)
        : "r"(x), "r"(y));
}

// MMA operands are warp-uniform registers.  The issuing warp therefore runs as a
// whole, on values the compiler knows to be uniform (parameters, block indexes,
// broadcasts from a fixed lane), and only the instruction itself is one lane's: with
// the whole loop inside one lane's branch every MMA took 97 cycles to issue, its
// descriptors moved to uniform registers one by one, instead of the 64 it runs for.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 r;\n\telect.sync r|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
constexpr uint32_t kNegateA = 1u << 13;  // instruction descriptor: D = -A B
// The lowest n of 32 bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint64_t step_desc(uint64_t d, uint32_t bytes) {
    return d + (bytes >> 4);  // no carry out of the address field: shared memory ends below 2^18
}
// Products of 128 x N tiles over D: `steps` steps of 16 of at most 4 NB.
template <int NB>
__device__ __forceinline__ void issue_rows(uint32_t d, uint64_t a, int ablock, uint64_t b, int bblock, uint32_t idesc, int steps) {
#pragma unroll
    for (int q = 0; q < 4 * NB; ++q)
        if (q < steps)
            umma_f16(d, step_desc(a, (q >> 2) * ablock + (q & 3) * 32), step_desc(b, (q >> 2) * bblock + (q & 3) * 32), idesc, q > 0);
}
// d (+)= a (tensor memory, steps [s0, s1) of 16 of its columns) times the tile b of those rows.  a's chunk
// of 32 columns lies in the first 16 of the columns of the chunk of scores that it came from.
template <int STEPS>
__device__ __forceinline__ void issue_sum(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int s0, int s1, bool accum) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        if (s >= s0 && s < s1) {
            umma_f16_ts(d, a + (s >> 1) * kTcChunk + (s & 1) * 8, step_desc(b, s * 2048), idesc, accum);
            accum = true;
        }
}

// Where rows see at most kBandExactKeys keys, p and d go to the tensor cores as two
// numbers of the I/O type, the second what the first leaves.
constexpr int kLow = 16;  // columns from the first numbers of a chunk to the second ones

// Two floats as a pair of T, and what the pair leaves of them.
template <typename T>
__device__ __forceinline__ uint32_t pack_low(float lo, float hi, uint32_t pair) {
    if constexpr (std::is_same<T, __half>::value) {
        __half2 h;
        memcpy(&h, &pair, 4);
        const float2 f = __half22float2(h);
        return pack2<T>(lo - f.x, hi - f.y);
    } else {
        return pack2<T>(lo - __uint_as_float(pair << 16), hi - __uint_as_float(pair & 0xffff0000u));
    }
}

// Lets a kernel have all of an SM's shared memory, once a thread and device (which
// also gives the thread its context: another thread may run a backward, and the
// maps' encoder asks for one).
constexpr int kMaxDynamicSmem = 225 << 10;
template <auto kernel>
cudaError_t allow_smem() {
    static thread_local unsigned long long done = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done >> dev & 1))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicSmem);
    if (e == cudaSuccess && dev < 64) done |= 1ull << dev;
    return e;
}

// cuTensorMapEncodeTiled from the driver (resolved once through the runtime).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn band_encode_tiled() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// [N][L][H][D] of 16-bit elements (strides in elements, 0 batch stride for one image) with boxes of
// 64 columns, `heads` heads and `rows` tokens, 128-byte swizzle, zeros outside.
inline bool make_map(CUtensorMap* map, int dtype, const void* base, int N, int L, int H, int D, long long batch, long long row,
                     int heads, int rows) {
    const EncodeTiledFn fn = band_encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(L),
                                static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(row) * 2,
                                   static_cast<cuuint64_t>(batch ? batch : row) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace dcn4
