// kv_cache.cuh -- cache formats: host checks, and decoding of stored rows to bf16.
//
// A group's scale is a power of two and a code has at most 4 significant bits, so a
// stored value is a bf16 number exactly: decoding places a code's exponent and mantissa
// bits in a bf16 and multiplies by a power of two (one packed multiply per two elements,
// nothing rounds).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace ssa {

// Bytes of one row of a cache.
__host__ __device__ constexpr int kv_row_bytes(int fmt, int d) {
    return fmt == SSA_KV_BF16 ? 2 * d : fmt == SSA_KV_E4M3 ? d : d / 2;
}

// Scale bytes E that a cache holds, beside 255 (a group that is not finite).
constexpr uint32_t kScaleMin = 16;
__host__ __device__ constexpr uint32_t kv_scale_max(int fmt) { return fmt == SSA_KV_E4M3 ? 134 : 140; }
__device__ __forceinline__ bool kv_bad_scale(int fmt, uint32_t E) { return E > kv_scale_max(fmt) && E != 255u; }

// Checks shared by the entry points that take a cache.
inline int check_cache(const char *fn, const ssa_kv_cache *c) {
    SSA_CHECK_ARG(c, "%s: null cache", fn);
    if (c->format != SSA_KV_BF16 && c->format != SSA_KV_E4M3 && c->format != SSA_KV_E2M1) {
        set_error("%s: unknown cache format %d", fn, c->format);
        return SSA_ERR_UNSUPPORTED;
    }
    if (c->d != 64 && c->d != 128) {
        set_error("%s: head dimension must be 64 or 128 (got %d)", fn, c->d);
        return SSA_ERR_UNSUPPORTED;
    }
    SSA_CHECK_ARG(c->B >= 1 && c->H_kv >= 1 && c->S >= 1, "%s: B, H_kv and S must be >= 1", fn);
    SSA_CHECK_ARG(c->B <= 65535 && c->H_kv <= 65535, "%s: B and H_kv must be <= 65535", fn);
    SSA_CHECK_ARG(c->k && c->v && (c->format == SSA_KV_BF16 || (c->k_scale && c->v_scale)), "%s: null cache buffer",
                  fn);
    SSA_CHECK_ARG(aligned16(c->k) && aligned16(c->v) &&
                      (c->format == SSA_KV_BF16 || (aligned16(c->k_scale) && aligned16(c->v_scale))),
                  "%s: cache buffers must be 16-byte aligned", fn);
    return SSA_OK;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// Packed bf16 products and sums.
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The factor that decode() multiplies by, in both halves, from a scale byte E.
//   e4m3: a code's 7 low bits shifted left by 4 are the bf16 of 2^-120 times its value
//         (subnormal codes become bf16 subnormals, which the multiply honours), so the
//         factor is 2^(E - 127 + 120): exponent field E + 120, at most 255
//   e2m1: decode gives the value itself; the factor is 2^(E - 127)
// E = 255 gives infinity; the group's codes are 0, and 0 * infinity is the NaN wanted.
template <int FMT>
__device__ __forceinline__ uint32_t kv_factor(uint32_t E) {
    const uint32_t f = FMT == SSA_KV_E4M3 ? min(E + 120u, 255u) : E;
    return (f << 7) * 0x10001u;
}

// Four e4m3 codes of a word -> bf16 pairs (bytes 0 and 2), (bytes 1 and 3), times factor.
__device__ __forceinline__ void decode_e4m3(uint32_t x, uint32_t factor, uint32_t &even, uint32_t &odd) {
    even = bf2_mul(((x & 0x007f007fu) << 4) | ((x & 0x00800080u) << 8), factor);
    odd = bf2_mul(((x >> 4) & 0x07f007f0u) | (x & 0x80008000u), factor);
}

// Four e2m1 codes in the low 16 bits of a word -> bf16 pairs (0, 1), (2, 3), times factor.
// The eight magnitudes 0 .5 1 1.5 2 3 4 6 are looked up a byte of their bf16 at a time.
__device__ __forceinline__ void decode_e2m1(uint32_t x, uint32_t factor, uint32_t &p01, uint32_t &p23) {
    const uint32_t idx = x & 0x7777u;
    const uint32_t hi = prmt(0x3f3f3f00u, 0x40404040u, idx), lo = prmt(0xc0800000u, 0xc0804000u, idx);
    p01 = bf2_mul(prmt(lo, hi, 0x5140u) | ((x << 12) & 0x8000u) | ((x << 24) & 0x80000000u), factor);
    p23 = bf2_mul(prmt(lo, hi, 0x7362u) | ((x << 4) & 0x8000u) | ((x << 16) & 0x80000000u), factor);
}

}  // namespace ssa
