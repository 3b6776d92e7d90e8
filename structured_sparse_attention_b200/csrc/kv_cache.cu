// kv_cache.cu -- filling a key/value cache and reading it back.
//
//   kv_append_kernel  queries, keys and values of a layer's projections: norm per head,
//                     position rotation, rounding to the cache's format, in one pass
//   kv_read_kernel    cache rows back to bf16
//
// The bytes they move are most of the work; the design keeps every access a full 16 (8, 4)
// bytes a lane over whole rows and computes a token's angles once for many heads.
#include "kv_cache.cuh"
#include "trace.h"

namespace ssa {
namespace {

constexpr int kThreads = 256;

struct Tokens {  // which cache row a token has
    const int32_t *ptr, *row0;
    int n_tokens, B, S;
};

// Sequence b and cache row of token t.  Returns 0 for a padding token, 1 for a valid row,
// -1 for a row outside the cache.  Whatever the lists hold, t is in [ptr[b], ptr[b+1]) of
// one sequence only, so two tokens never get the same row.
__device__ __forceinline__ int find_row(const Tokens &k, int t, int &b, int &row) {
    b = 0;
    if (t >= k.n_tokens) return 0;
    if (k.B > 1) {
        int lo = 0, hi = k.B;  // first b with ptr[b + 1] > t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(k.ptr + mid + 1) <= t) lo = mid + 1;
            else hi = mid;
        }
        if (lo == k.B) return 0;
        b = lo;
    }
    const int p0 = __ldg(k.ptr + b), p1 = __ldg(k.ptr + b + 1);
    if (t < p0 || t >= p1) return 0;
    const int r0 = __ldg(k.row0 + b);
    const long long r = static_cast<long long>(r0) + (t - p0);
    row = static_cast<int>(r);
    return p0 >= 0 && r0 >= 0 && r < k.S ? 1 : -1;
}

// One block looks over the descriptors.
__device__ void check_tokens(const Tokens &k, int32_t *status) {
    for (int b = threadIdx.x; b < k.B; b += blockDim.x) {
        const int p0 = __ldg(k.ptr + b), p1 = __ldg(k.ptr + b + 1), r0 = __ldg(k.row0 + b);
        if (p0 < 0 || p1 < p0 || p1 > k.n_tokens || r0 < 0 || static_cast<long long>(r0) + p1 - p0 > k.S)
            report(status, SSA_ERR_INVALID);
    }
}

struct AppendParams {
    Tokens tok;
    int n_pad, Hq, Hkv, chunk;  // tokens rounded up to whole warps; rows (heads) a unit takes
    const uint16_t *q, *k, *v;
    int64_t qt, qh, kt, kh, vt, vh;
    uint16_t *qo, *ko, *vo;
    int64_t qot, qoh, kot, koh, vot, voh;
    const int32_t *pos;
    const double *freqs;
    const float *qw, *kw;
    float eps;
    uint8_t *ck, *cv, *sk, *sv;
    int32_t *status;
};

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }

// bf16 pairs <-> packed fp32 pairs
__device__ __forceinline__ uint64_t widen(uint32_t w) {
    return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint32_t narrow(uint64_t x) {
    float lo, hi;
    f2_unpack(x, lo, hi);
    return pack2(lo, hi);
}

__device__ __forceinline__ uint4 narrow8(const uint64_t *x) {
    return make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
}

// The largest |x| of four pairs; a NaN stays on top.
__device__ __forceinline__ float amax8(const uint64_t *x) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(x[i], lo, hi);
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(lo)), "f"(fabsf(hi)));
    }
    return m;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Scale byte of a group from the bits of its largest |x| (a NaN or an infinity if it holds
// one): the smallest e with |x| <= M 2^e, M = 1.75 * 2^8 or 1.5 * 2^2.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255u;
    const int exp = static_cast<int>(amax >> 23);
    const uint32_t man = amax & 0x7fffffu;
    const int E = FMT == SSA_KV_E4M3 ? exp - 8 + (man > 0x600000u) : exp - 2 + (man > 0x400000u);
    return static_cast<uint32_t>(min(max(E, static_cast<int>(kScaleMin)), static_cast<int>(kv_scale_max(FMT))));
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ uint32_t to_e2m1x8(const float *x) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, e;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, e};\n\t}"
        : "=r"(d)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return d;
}

// The lanes of a unit hold one row: lane l the elements 8l .. 8l+7 of each half of the row,
// so that both kinds of rotated pair lie within a lane and a group of 32 within 4 lanes.
// A row of the cache and, where wanted, the bf16 values that it stands for.
template <int D, int FMT>
__device__ __forceinline__ void store_row(const uint64_t (&x)[8], int l, bool write, uint8_t *row, uint8_t *srow,
                                          uint16_t *out) {
    uint4 val[2];
    if constexpr (FMT == SSA_KV_BF16) {
        val[0] = narrow8(x);
        val[1] = narrow8(x + 4);
        if (write) {
            *reinterpret_cast<uint4 *>(row + 16 * l) = val[0];
            *reinterpret_cast<uint4 *>(row + D + 16 * l) = val[1];
        }
    } else {
        uint32_t E[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float amax = amax8(x + 4 * hf);
            amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            E[hf] = scale_byte<FMT>(__float_as_uint(amax));
            // times 2^(127 - E): exact; a group that is not finite becomes codes 0
            const bool bad = E[hf] == 255u;
            const float inv = __uint_as_float((bad ? 0u : 254u - E[hf]) << 23);
            const uint64_t inv2 = f2_pack(inv, inv);
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(x[4 * hf + i], inv2), y[2 * i], y[2 * i + 1]);
            const uint32_t f = kv_factor<FMT>(E[hf]);
            if constexpr (FMT == SSA_KV_E4M3) {
                uint2 c = make_uint2(to_e4m3x4(y[0], y[1], y[2], y[3]), to_e4m3x4(y[4], y[5], y[6], y[7]));
                if (bad) c = make_uint2(0, 0);
                if (write) *reinterpret_cast<uint2 *>(row + hf * (D / 2) + 8 * l) = c;
                if (out) {
                    uint32_t a, b;
                    decode_e4m3(c.x, f, a, b);
                    val[hf].x = prmt(a, b, 0x5410u);
                    val[hf].y = prmt(a, b, 0x7632u);
                    decode_e4m3(c.y, f, a, b);
                    val[hf].z = prmt(a, b, 0x5410u);
                    val[hf].w = prmt(a, b, 0x7632u);
                }
            } else {
                uint32_t c = to_e2m1x8(y);
                if (bad) c = 0;
                if (write) *reinterpret_cast<uint32_t *>(row + hf * (D / 4) + 4 * l) = c;
                if (out) {
                    decode_e2m1(c, f, val[hf].x, val[hf].y);
                    decode_e2m1(c >> 16, f, val[hf].z, val[hf].w);
                }
            }
        }
        if constexpr (D == 128) {  // groups 0, 1 of a half are the lanes 0-3 and 4-7
            const uint32_t e = E[0] | (E[1] << 16);
            const uint32_t all = e | (__shfl_down_sync(0xffffffffu, e, 4) << 8);
            if (write && l == 0) *reinterpret_cast<uint32_t *>(srow) = all;
        } else {
            if (write && l == 0) *reinterpret_cast<uint16_t *>(srow) = static_cast<uint16_t>(E[0] | (E[1] << 8));
        }
    }
    if (out && write) {
        *reinterpret_cast<uint4 *>(out + 8 * l) = val[0];
        *reinterpret_cast<uint4 *>(out + D / 2 + 8 * l) = val[1];
    }
}

// Sine and cosine of a whole number of turns, in fp64 until their one rounding to fp32: the
// nearest quarter turn is taken out, the rest, at most pi / 4, goes through the Taylor sums to
// x^11 and x^10 (the next terms are below 2^-36 and 2^-32).  The reduction itself is exact, so
// position 2^20 still has its angle to 2^-33 of a turn, and keys near a border between two codes
// fall as the exact ones do.
__device__ __forceinline__ void sincos_turn(double turn, float &s, float &c) {
    turn -= rint(turn);
    const double k = rint(4.0 * turn);
    const double x = (turn - 0.25 * k) * 6.283185307179586477, x2 = x * x;
    double u = fma(x2, -1.0 / 39916800, 1.0 / 362880), v = fma(x2, -1.0 / 3628800, 1.0 / 40320);
    u = fma(x2, u, -1.0 / 5040);
    v = fma(x2, v, -1.0 / 720);
    u = fma(x2, u, 1.0 / 120);
    v = fma(x2, v, 1.0 / 24);
    u = fma(x2, u, -1.0 / 6);
    v = fma(x2, v, -0.5);
    const float sf = static_cast<float>(fma(x * x2, u, x)), cf = static_cast<float>(fma(x2, v, 1.0));
    const int q = static_cast<int>(k) & 3;
    const float a = (q & 1) ? cf : sf, b = (q & 1) ? sf : cf;
    s = (q & 2) ? -a : a;
    c = (q == 1 || q == 2) ? -b : b;
}

// D / 16 lanes (a unit) take one token and `chunk` of its H_q + 2 H_kv rows; the tokens of a
// warp's units are neighbours and share the rows' heads, so cache rows are written in runs
// and all branches on the head are uniform.  A lane's part of the next rows travels by
// cp.async into slots of its own in shared memory, kAhead rows ahead: what is in flight
// takes no registers and needs no barrier.  Arithmetic is on packed pairs.
//
// 16384 tokens of 32 + 2 x 8 heads, d = 64, with k_out and v_out: to e4m3 49 us, 4.5 TB/s moved, 68 %
// of the card's copy rate; to bf16 47 us, 5.0 TB/s; to e2m1 50 us, 4.2 TB/s.  Nothing is full: DRAM is
// active 41 % of the time and the schedulers issue in half of the cycles, with the 4 warps each
// that two CTAs of 106 registers a thread leave; 768 CTAs on 296 places are 2.6 waves.  With a
// register prefetch of the rows in place of cp.async it took 66 us.
constexpr int kAhead = 4;

__device__ __forceinline__ void copy16(void *dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

template <int D, int FMT, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int LPR = D / 16;
    const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
    const int l = threadIdx.x % LPR;
    const long long c = unit / p.n_pad;
    const int t = static_cast<int>(unit - c * p.n_pad);
    const int HT = p.Hq + 2 * p.Hkv;
    if (blockIdx.x == 0) check_tokens(p.tok, p.status);
    if (c * p.chunk >= HT) return;  // whole warps: n_pad is a multiple of a warp's units
    const int r_begin = static_cast<int>(c) * p.chunk, r_end = min(HT, r_begin + p.chunk);

    __shared__ uint4 s_in[kAhead][2][kThreads];
    const bool there = t < p.tok.n_tokens;
    const auto load = [&](int r, int slot) {  // zeros for a row that is not there
        const uint16_t *src = r < p.Hq ? p.q + t * p.qt + r * p.qh
                              : r < p.Hq + p.Hkv ? p.k + t * p.kt + (r - p.Hq) * p.kh
                                                 : p.v + t * p.vt + (r - p.Hq - p.Hkv) * p.vh;
        const bool valid = there && r < r_end;
        if (!valid) src = p.k;
        copy16(&s_in[slot][0][threadIdx.x], src + 8 * l, valid);
        copy16(&s_in[slot][1][threadIdx.x], src + D / 2 + 8 * l, valid);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(r_begin + u, u);

    int b, row = 0;
    bool ok = find_row(p.tok, t, b, row) == 1;
    int P = row;
    if (p.pos && ok) {
        P = __ldg(p.pos + t);
        if (P < 0) {
            ok = false;
            if (l == 0) report(p.status, SSA_ERR_INVALID);
        }
    }
    uint64_t cs[4], sn[4];  // of the lane's 8 rotated pairs
    if (p.freqs && r_begin < p.Hq + p.Hkv) {
        float c1[8], s1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pair = INTER ? (i < 4 ? 4 * l + i : D / 4 + 4 * l + i - 4) : 8 * l + i;
            double turn = static_cast<double>(P) * (__ldg(p.freqs + pair) * 0.15915494309189533577);
            sincos_turn(turn, s1[i], c1[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cs[i] = f2_pack(c1[2 * i], c1[2 * i + 1]);
            sn[i] = f2_pack(s1[2 * i], s1[2 * i + 1]);
        }
    }
    uint64_t w[8];
    int w_kind = -1;
    const auto work = [&](int r, int slot) {
        const uint4 raw[2] = {s_in[slot][0][threadIdx.x], s_in[slot][1][threadIdx.x]};
        load(r + kAhead, slot);
        const int kind = r < p.Hq ? 0 : r < p.Hq + p.Hkv ? 1 : 2;
        uint64_t x[8] = {widen(raw[0].x), widen(raw[0].y), widen(raw[0].z), widen(raw[0].w),
                         widen(raw[1].x), widen(raw[1].y), widen(raw[1].z), widen(raw[1].w)};
        const float *weight = kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr;
        if (weight) {
            if (kind != w_kind) {
                w_kind = kind;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = f2_pack(__ldg(weight + 8 * l + 2 * i), __ldg(weight + 8 * l + 2 * i + 1));
                    w[4 + i] = f2_pack(__ldg(weight + D / 2 + 8 * l + 2 * i), __ldg(weight + D / 2 + 8 * l + 2 * i + 1));
                }
            }
            uint64_t s2 = f2_mul(x[0], x[0]), s3 = f2_mul(x[1], x[1]);
#pragma unroll
            for (int i = 2; i < 8; i += 2) {
                s2 = f2_fma(x[i], x[i], s2);
                s3 = f2_fma(x[i + 1], x[i + 1], s3);
            }
            float s0, s1;
            f2_unpack(f2_add(s2, s3), s0, s1);
            float ss = s0 + s1;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rs = __frsqrt_rn(fmaf(ss, 1.0f / D, p.eps));
            const uint64_t rs2 = f2_pack(rs, rs);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = f2_mul(f2_mul(x[i], rs2), w[i]);
        }
        if (kind < 2 && p.freqs) {
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float a, z, c0[2], s0[2];
                    f2_unpack(x[i], a, z);
                    f2_unpack(cs[i / 2], c0[0], c0[1]);
                    f2_unpack(sn[i / 2], s0[0], s0[1]);
                    x[i] = f2_pack(fmaf(a, c0[i & 1], -(z * s0[i & 1])), fmaf(z, c0[i & 1], a * s0[i & 1]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t a = x[i], z = x[4 + i];
                    x[i] = f2_fma(a, cs[i], f2_neg(f2_mul(z, sn[i])));
                    x[4 + i] = f2_fma(z, cs[i], f2_mul(a, sn[i]));
                }
            }
        }
        if (kind == 0) {
            if (ok) {
                uint16_t *dst = p.qo + t * p.qot + r * p.qoh;
                *reinterpret_cast<uint4 *>(dst + 8 * l) = narrow8(x);
                *reinterpret_cast<uint4 *>(dst + D / 2 + 8 * l) = narrow8(x + 4);
            }
        } else {
            const int g = r - p.Hq - (kind - 1) * p.Hkv;
            const size_t at = (static_cast<size_t>(b) * p.Hkv + g) * p.tok.S + (ok ? row : 0);
            uint16_t *out = kind == 1 ? p.ko : p.vo;
            if (out) out += kind == 1 ? t * p.kot + g * p.koh : t * p.vot + g * p.voh;
            store_row<D, FMT>(x, l, ok, (kind == 1 ? p.ck : p.cv) + at * kv_row_bytes(FMT, D),
                              (kind == 1 ? p.sk : p.sv) + at * (D / SSA_KV_GROUP), out);
        }
    };
#pragma unroll 1
    for (int r = r_begin, slot = 0; r < r_end; ++r, slot = (slot + 1) % kAhead) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        work(r, slot);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

struct ReadParams {
    Tokens tok;
    int Hkv;
    const uint8_t *ck, *cv, *sk, *sv;
    uint16_t *ko, *vo;
    int64_t kot, koh, vot, voh;
    int32_t *status;
};

// A lane decodes 8 elements (one 16-byte store) of each of kReadAhead tokens, whose loads are all
// under way before the first is used; a CTA takes one head of the keys or of the values.
//
// 65536 tokens of 8 heads, d = 128: bf16 80 us, 6.7 TB/s moved; e4m3 65 us, 6.3 TB/s, 96 % of the card's
// copy rate; e2m1 71 us, 4.8 TB/s.  bf16 and e4m3 are bound by memory.  e2m1 is bound by
// instructions: 3 x 104000 tokens take 340 us, 4.0 TB/s moved (3.2 of them writes, where a fill of
// memory reaches 4.0), with 84 % of the issue slots full: the descriptor search of each lane and
// token and the decoding, for 16 bytes written.
constexpr int kReadAhead = 4;

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int LPR = D / 8, RPP = kThreads / LPR;
    const int l = threadIdx.x % LPR, g = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    if (blockIdx.x == 0 && g == 0 && !is_v) check_tokens(p.tok, p.status);
    const uint8_t *codes = is_v ? p.cv : p.ck, *scales = is_v ? p.sv : p.sk;
    uint16_t *out = is_v ? p.vo : p.ko;
    const int64_t ts = is_v ? p.vot : p.kot, hs = is_v ? p.voh : p.koh;
    const int t0 = blockIdx.x * (RPP * kReadAhead) + threadIdx.x / LPR;
    bool ok[kReadAhead];
    uint4 raw[kReadAhead];
    uint32_t E[kReadAhead];
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
        int b, row = 0;
        ok[u] = find_row(p.tok, t0 + u * RPP, b, row) == 1;
        if (!ok[u]) continue;
        const size_t at = (static_cast<size_t>(b) * p.Hkv + g) * p.tok.S + row;
        const uint8_t *src = codes + at * kv_row_bytes(FMT, D);
        if constexpr (FMT == SSA_KV_BF16) {
            raw[u] = __ldg(reinterpret_cast<const uint4 *>(src) + l);
        } else if constexpr (FMT == SSA_KV_E4M3) {
            const uint2 c = __ldg(reinterpret_cast<const uint2 *>(src) + l);
            raw[u].x = c.x;
            raw[u].y = c.y;
        } else {
            raw[u].x = __ldg(reinterpret_cast<const uint32_t *>(src) + l);
        }
        if constexpr (FMT != SSA_KV_BF16) E[u] = __ldg(scales + at * (D / SSA_KV_GROUP) + l / 4);
    }
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
        if (!ok[u]) continue;
        if constexpr (FMT != SSA_KV_BF16)
            if (kv_bad_scale(FMT, E[u])) report(p.status, SSA_ERR_INVALID);
        uint4 v = raw[u];
        if constexpr (FMT == SSA_KV_E4M3) {
            const uint32_t f = kv_factor<FMT>(E[u]);
            uint32_t a, b;
            decode_e4m3(raw[u].x, f, a, b);
            v.x = prmt(a, b, 0x5410u);
            v.y = prmt(a, b, 0x7632u);
            decode_e4m3(raw[u].y, f, a, b);
            v.z = prmt(a, b, 0x5410u);
            v.w = prmt(a, b, 0x7632u);
        } else if constexpr (FMT == SSA_KV_E2M1) {
            const uint32_t f = kv_factor<FMT>(E[u]);
            decode_e2m1(raw[u].x, f, v.x, v.y);
            decode_e2m1(raw[u].x >> 16, f, v.z, v.w);
        }
        const int64_t t = t0 + u * RPP;
        *reinterpret_cast<uint4 *>(out + t * ts + g * hs + 8 * l) = v;
    }
}

template <int D, int FMT>
int launch_append(const AppendParams &p, bool inter, cudaStream_t s) {
    const long long units = static_cast<long long>(p.n_pad) * ((p.Hq + 2 * p.Hkv + p.chunk - 1) / p.chunk);
    const long long grid = (units * (D / 16) + kThreads - 1) / kThreads;
    SSA_CHECK_ARG(grid <= 0x7fffffffLL, "sparse_kv_append: too many tokens");
    if (inter) kv_append_kernel<D, FMT, true><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    else kv_append_kernel<D, FMT, false><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    SSA_LAUNCH_CHECK();
    return SSA_OK;
}

template <int D, int FMT>
int launch_read(const ReadParams &p, cudaStream_t s) {
    constexpr int per_cta = kThreads / (D / 8) * kReadAhead;
    kv_read_kernel<D, FMT><<<dim3((p.tok.n_tokens + per_cta - 1) / per_cta, p.Hkv, 2), kThreads, 0, s>>>(p);
    SSA_LAUNCH_CHECK();
    return SSA_OK;
}

bool good_rows(const ssa_rows &r) {
    return aligned16(r.ptr) && r.token_stride >= 0 && r.head_stride >= 0 && r.token_stride % 8 == 0 &&
           r.head_stride % 8 == 0;
}

// An output's rows must not share memory: heads within tokens or tokens within heads.
bool good_out(const ssa_rows &r, int64_t n, int64_t heads, int d) {
    const int64_t ts = n > 1 ? r.token_stride : 0, hs = heads > 1 ? r.head_stride : 0;
    if (!r.ptr) return true;
    const bool token_major = (n == 1 || ts >= (heads - 1) * hs + d) && (heads == 1 || hs >= d);
    const bool head_major = (heads == 1 || hs >= (n - 1) * ts + d) && (n == 1 || ts >= d);
    return good_rows(r) && (token_major || head_major);
}

}  // namespace
}  // namespace ssa

using namespace ssa;

extern "C" int sparse_kv_append(const ssa_kv_cache *cache, const ssa_kv_append_args *a, int32_t *dev_status,
                                void *stream) {
    ssa::TraceRange trace_range("sparse_kv_append");
    if (const int rc = check_cache("sparse_kv_append", cache)) return rc;
    SSA_CHECK_ARG(a, "sparse_kv_append: null arguments");
    if (a->n_tokens == 0) return SSA_OK;  // the views of no tokens may have no storage
    SSA_CHECK_ARG(a->k.ptr && a->v.ptr && a->tok_ptr && a->row0, "sparse_kv_append: null pointer argument");
    SSA_CHECK_ARG(a->n_tokens >= 0 && a->H_q >= 0 && a->H_q <= 65535,
                  "sparse_kv_append: n_tokens must be >= 0 and H_q in [0, 65535]");
    SSA_CHECK_ARG((a->H_q > 0) == (a->q.ptr != nullptr) && (a->H_q > 0) == (a->q_out.ptr != nullptr),
                  "sparse_kv_append: q and q_out go with H_q > 0");
    SSA_CHECK_ARG((a->k_out.ptr != nullptr) == (a->v_out.ptr != nullptr),
                  "sparse_kv_append: k_out and v_out go together");
    SSA_CHECK_ARG(good_rows(a->q) && good_rows(a->k) && good_rows(a->v) && good_rows(a->q_out) &&
                      good_rows(a->k_out) && good_rows(a->v_out),
                  "sparse_kv_append: rows must be 16-byte aligned with strides in multiples of 8 elements");
    SSA_CHECK_ARG(!(a->q_weight || a->k_weight) || (a->eps > 0.0f && a->eps < 1e30f),
                  "sparse_kv_append: eps must be positive and finite");
    SSA_CHECK_ARG(good_out(a->q_out, a->n_tokens, a->H_q, cache->d) &&
                      good_out(a->k_out, a->n_tokens, cache->H_kv, cache->d) &&
                      good_out(a->v_out, a->n_tokens, cache->H_kv, cache->d),
                  "sparse_kv_append: rows of an output overlap");
    const int d = cache->d, per_warp = 32 / (d / 16);
    SSA_CHECK_ARG(a->n_tokens <= 0x7fffffff - 32, "sparse_kv_append: too many tokens");
    AppendParams p{};
    p.tok = {a->tok_ptr, a->row0, a->n_tokens, cache->B, cache->S};
    p.n_pad = (a->n_tokens + per_warp - 1) / per_warp * per_warp;
    p.Hq = a->H_q;
    p.Hkv = cache->H_kv;
    // Rows a unit takes: as many as leave 32 warps for each SM (a token's angles are then
    // computed once for up to 16 rows), one where there are few tokens.  With 1 and 16 rows:
    // 16 sequences of up to 13 tokens (118) of 32 + 2 x 8 heads 5.2 and 16.0 us, 16384 tokens 112 and 49 us.
    const int HT = p.Hq + 2 * p.Hkv;
    p.chunk = 16;
    while (p.chunk > 1 && static_cast<long long>(p.n_pad) * ((HT + p.chunk - 1) / p.chunk) / per_warp < 148 * 32)
        p.chunk >>= 1;
    p.q = static_cast<const uint16_t *>(a->q.ptr);
    p.k = static_cast<const uint16_t *>(a->k.ptr);
    p.v = static_cast<const uint16_t *>(a->v.ptr);
    p.qt = a->q.token_stride, p.qh = a->q.head_stride;
    p.kt = a->k.token_stride, p.kh = a->k.head_stride;
    p.vt = a->v.token_stride, p.vh = a->v.head_stride;
    p.qo = static_cast<uint16_t *>(a->q_out.ptr);
    p.ko = static_cast<uint16_t *>(a->k_out.ptr);
    p.vo = static_cast<uint16_t *>(a->v_out.ptr);
    p.qot = a->q_out.token_stride, p.qoh = a->q_out.head_stride;
    p.kot = a->k_out.token_stride, p.koh = a->k_out.head_stride;
    p.vot = a->v_out.token_stride, p.voh = a->v_out.head_stride;
    p.pos = a->pos;
    p.freqs = a->freqs;
    p.qw = a->q_weight;
    p.kw = a->k_weight;
    p.eps = a->eps;
    p.ck = static_cast<uint8_t *>(cache->k);
    p.cv = static_cast<uint8_t *>(cache->v);
    p.sk = cache->k_scale;
    p.sv = cache->v_scale;
    p.status = dev_status;
    const bool inter = a->interleaved != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d == 64) {
        if (cache->format == SSA_KV_BF16) return launch_append<64, SSA_KV_BF16>(p, inter, s);
        if (cache->format == SSA_KV_E4M3) return launch_append<64, SSA_KV_E4M3>(p, inter, s);
        return launch_append<64, SSA_KV_E2M1>(p, inter, s);
    }
    if (cache->format == SSA_KV_BF16) return launch_append<128, SSA_KV_BF16>(p, inter, s);
    if (cache->format == SSA_KV_E4M3) return launch_append<128, SSA_KV_E4M3>(p, inter, s);
    return launch_append<128, SSA_KV_E2M1>(p, inter, s);
}

extern "C" int sparse_kv_read(const ssa_kv_cache *cache, int n_tokens, const int32_t *tok_ptr, const int32_t *row0,
                              const ssa_rows *k_out, const ssa_rows *v_out, int32_t *dev_status, void *stream) {
    ssa::TraceRange trace_range("sparse_kv_read");
    if (const int rc = check_cache("sparse_kv_read", cache)) return rc;
    if (n_tokens == 0) return SSA_OK;  // the views of no tokens may have no storage
    SSA_CHECK_ARG(tok_ptr && row0 && k_out && v_out && k_out->ptr && v_out->ptr,
                  "sparse_kv_read: null pointer argument");
    SSA_CHECK_ARG(n_tokens >= 0 && n_tokens <= 0x7fffffff - 1024, "sparse_kv_read: n_tokens out of range");
    SSA_CHECK_ARG(good_rows(*k_out) && good_rows(*v_out),
                  "sparse_kv_read: rows must be 16-byte aligned with strides in multiples of 8 elements");
    SSA_CHECK_ARG(good_out(*k_out, n_tokens, cache->H_kv, cache->d) && good_out(*v_out, n_tokens, cache->H_kv, cache->d),
                  "sparse_kv_read: rows of an output overlap");
    ReadParams p{};
    p.tok = {tok_ptr, row0, n_tokens, cache->B, cache->S};
    p.Hkv = cache->H_kv;
    p.ck = static_cast<const uint8_t *>(cache->k);
    p.cv = static_cast<const uint8_t *>(cache->v);
    p.sk = cache->k_scale;
    p.sv = cache->v_scale;
    p.ko = static_cast<uint16_t *>(k_out->ptr);
    p.vo = static_cast<uint16_t *>(v_out->ptr);
    p.kot = k_out->token_stride, p.koh = k_out->head_stride;
    p.vot = v_out->token_stride, p.voh = v_out->head_stride;
    p.status = dev_status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cache->d == 64) {
        if (cache->format == SSA_KV_BF16) return launch_read<64, SSA_KV_BF16>(p, s);
        if (cache->format == SSA_KV_E4M3) return launch_read<64, SSA_KV_E4M3>(p, s);
        return launch_read<64, SSA_KV_E2M1>(p, s);
    }
    if (cache->format == SSA_KV_BF16) return launch_read<128, SSA_KV_BF16>(p, s);
    if (cache->format == SSA_KV_E4M3) return launch_read<128, SSA_KV_E4M3>(p, s);
    return launch_read<128, SSA_KV_E2M1>(p, s);
}
