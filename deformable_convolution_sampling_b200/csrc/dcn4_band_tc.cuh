// dcn4_band_tc.cuh — what the band attention's tensor-core kernels share: operand
// tiles of 128 rows in the 128-byte swizzled layout, products whose first operand
// is in tensor memory, and tensor-memory loads and stores by a thread per row.
//
// Operand tile: 128 rows (queries or keys) of D entries in blocks of 64 columns;
// row r of a block is 128 bytes at r * 128, its 16-byte pieces permuted by r mod 8.
// As a K-major operand (contraction over D) a step of 16 entries moves 32 bytes,
// as an M/N-major one (contraction over the rows) a step of 16 rows moves 2048
// bytes and the blocks are kTcBlock apart.  Rows past a sequence and entries past
// D are zeros: a TMA box would bring what lies there, and 0 times an infinity is
// not 0, so the tiles are filled with 16-byte cp.async, which write zeros instead.
#pragma once

#include <type_traits>

#include "dcn4_band_parts.cuh"
#include "dcn4_common.cuh"
#include "dcn4_tcgen05.cuh"

namespace dcn4 {
namespace tc {

constexpr int kTcRows = 128;                 // rows of a tile: the MMA's M, TMEM's lanes
constexpr int kTcBlock = kTcRows * 128;      // bytes of a block of 64 columns
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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One tile of `rows` (a multiple of 8) rows by 128 threads: row(r) gives a row's address, or NULL for
// zeros; `safe` is any valid address of the tensor.  A warp reads 256 (D > 64) or
// 128 bytes of neighbouring pieces of a row.
template <typename T, int NB, typename Row>
__device__ __forceinline__ void load_operand(uint32_t dst, int D, int rows, const T* safe, Row row, int tid) {
    constexpr int P = 8 * NB;  // pieces of a padded row
    const int piece = tid % P, col = piece * 8;
    const bool in = col < D;
    if (col >= (D + 15) / 16 * 16) return;  // no product reads these
    const uint32_t at = dst + (piece / 8) * kTcBlock;
    for (int r = tid / P; r < rows; r += 128 / P) {
        const T* src = row(r);
        const bool on = in && src;
        cp16(at + r * 128 + (((piece & 7) ^ (r & 7)) << 4), on ? src + col : safe, on);
    }
}

// Products of 128 x N tiles over D: D rounded up to steps of 16.
__device__ __forceinline__ void issue_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int steps) {
    for (int q = 0; q < steps; ++q) {
        const uint32_t off = (q >> 2) * kTcBlock + (q & 3) * 32;
        umma_f16(d, umma_desc_sw128(a + off, 16, 1024), umma_desc_sw128(b + off, 16, 1024), idesc, q > 0);
    }
}
// d (+)= a (tensor memory, K steps of 16 rows [s0, s1)) times the tile b of those rows.
__device__ __forceinline__ void issue_sum(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int s0, int s1, bool accum) {
    for (int s = s0; s < s1; ++s)
        umma_f16_ts(d, a + s * 8, umma_desc_sw128(b + s * 2048, kTcBlock, 1024), idesc, accum || s > s0);
}

}  // namespace tc
}  // namespace dcn4
