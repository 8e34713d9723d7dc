// Pieces shared by the token-sequence attention kernels (prompt.cu, pages_attention.cu):
// the softmax of one 128-key score tile in a thread's registers, 16-bit type traits and
// TMA wrappers.  A score tile is 128 query rows x 128 keys in TMEM, one row per thread.
#pragma once

#include "ptx.cuh"

namespace sdv2 {

// All 32 lanes wait; the warp proceeds only if every lane saw the phase complete, so
// the .sync.aligned tcgen05 ops that follow stay warp-uniform.
__device__ __forceinline__ bool warp_wait_all(uint64_t *bar, uint32_t parity, volatile uint32_t *abort,
                                              uint32_t *status, uint32_t code) {
    const bool ok = mbar_wait(bar, parity, abort, status, code);
    return __all_sync(0xffffffffu, ok);
}

// 3-D tile load global -> shared, completion counted in bytes on `bar`.  c0 (innermost)
// must be a multiple of 16 bytes / element size.
__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                            int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Instruction descriptor for kind::f16 with an fp32 accumulator and A and B both bf16
// (HALF false) or both fp16 (HALF true).
template <bool HALF>
__host__ __device__ constexpr uint32_t idesc_16_f32(int m, int n, int a_mn, int b_mn) {
    return (1u << 4) | ((HALF ? 0u : 1u) << 7) | ((HALF ? 0u : 1u) << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// Two fp32 -> packed fp16 or bf16 pair (lo in bits 0..15), round to nearest even.
template <bool HALF>
__device__ __forceinline__ uint32_t pack_16x2(float lo, float hi) {
    if constexpr (HALF) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        return pack_bf16x2(lo, hi);
    }
}

constexpr float kCoreRescale = 8.0f;   // log2 units: the running maximum moves only when a tile exceeds it by > 2^8

// The 128 scores of this thread's row, raw fp32 bits.
struct ScoreRow {
    uint32_t s[4][32];
};

__device__ __forceinline__ void load_scores(uint32_t s_tmem, ScoreRow &r) {
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) tmem_ld32(s_tmem + cb * 32, r.s[cb]);
    tmem_wait_ld_bind(r.s[0]);
#pragma unroll
    for (int cb = 1; cb < 4; ++cb) reg_bind(r.s[cb]);
}

// Keys at columns >= valid leave the softmax: their scores, whatever they hold (keys past
// the sequence may be anything, NaN included), become -inf.
__device__ __forceinline__ void mask_scores(ScoreRow &r, int valid) {
#pragma unroll
    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (cb * 32 + i >= valid) r.s[cb][i] = 0xff800000u;
}

// Largest score of the row: four chains of three-input maxima.
__device__ __forceinline__ float max_score(const ScoreRow &r) {
    float m4[4];
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) {
        float m = __uint_as_float(r.s[cb][0]);
#pragma unroll
        for (int i = 1; i < 31; i += 2)
            m = fmax3(m, __uint_as_float(r.s[cb][i]), __uint_as_float(r.s[cb][i + 1]));
        m4[cb] = fmaxf(m, __uint_as_float(r.s[cb][31]));
    }
    return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
}

// P = 2^(s * scale_log2 - m), rounded to 16 bits for the tensor cores into TMEM columns
// [0, 64) of the row's score region; returns the row sum of the unrounded values.  The
// rounding of P (half a step, relative) is the only one between the scores and the output's
// own; the sum, the maximum and the accumulator are fp32.
template <bool HALF>
__device__ __forceinline__ float exp_store(const ScoreRow &r, float scale_log2, float neg_m, uint32_t s_tmem) {
    const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
    const uint64_t negm2 = f2_pack(neg_m, neg_m);
    uint64_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = 0ull;
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint64_t x = f2_fma(f2_pack(__uint_as_float(r.s[cb][2 * i]), __uint_as_float(r.s[cb][2 * i + 1])),
                                      scale2, negm2);
            float x0, x1;
            f2_unpack(x, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            acc[i & 3] = f2_add(acc[i & 3], f2_pack(p0, p1));
            pk[i] = pack_16x2<HALF>(p0, p1);
        }
        tmem_st16(s_tmem + cb * 16, pk);
    }
    float a0, a1;
    f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
    return a0 + a1;
}

// Multiply this thread's row of an accumulator (D fp32 columns) by alpha.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t o_tmem, float alpha) {
#pragma unroll
    for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t r[32];
        tmem_ld32(o_tmem + cb * 32, r);
        tmem_wait_ld_bind(r);
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
        tmem_st32(o_tmem + cb * 32, r);
    }
}

// Rows [valid, 128) of a V tile (D / 64 sub-tiles of 128 rows x 128 bytes) set to zero by
// one warp: a masked key's probability is 0, and 0 times what lies past the sequence (NaN
// and infinities included) must add nothing.  Fenced for the tensor core.
template <int D>
__device__ __forceinline__ void zero_tail_rows(uint8_t *tile, int valid, int lane) {
    const int chunks = (128 - valid) * 8;                 // 16-byte chunks of one sub-tile
#pragma unroll
    for (int kb = 0; kb < D / 64; ++kb)
        for (int i = lane; i < chunks; i += 32)
            *reinterpret_cast<uint4 *>(tile + kb * (128 * 128) + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
    __syncwarp();
}

}  // namespace sdv2
