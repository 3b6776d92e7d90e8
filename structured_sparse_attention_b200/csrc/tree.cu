// tree.cu -- attention of drafted trees over a key/value cache, under the extended mask.
//
// One (sequence, KV head) is one problem: its rows are the tree's nodes for every query
// head of the group (row = head of the group * nodes + node), its keys the union list of
// the group (tree_lists.cu) cut at the sequence's length, then the nodes' own cache rows.
// Each key and value is read once for all rows; which row retains it is a bit:
//   committed key j, row (h, n):  bit t_n of the 64-bit window of D_h's bitmap at
//                                 o = len - j  (o + t_n is a diagonal), or j in C_h
//   node a:                       a is n or an ancestor, and t_n - t_a in D_h or p_a in C_h
// This file takes up to 32 rows a KV head (single tokens, small trees), tree_wide.cu more.
//
// Products run on the tensor cores by mma.sync (m16n8k16, fp32 accumulation).  With 32 rows or
// fewer a 128-row tensor-memory tile would be mostly empty, and a step's time goes into
// gathering and decoding the rows; fragments of mma.sync are filled from the gathered rows
// as each warp has them, without a barrier between warps.  bf16 caches multiply as bf16, the
// codes of e4m3 and e2m1 as fp16, which holds them exactly times their scale; steps with a group
// too small for that multiply as bf16 too.  16 sequences x 8 KV heads over lists of 900 e4m3 keys,
// 4 / 16 / 32 rows: 18.2 / 19.9 / 27.1 us, with values of deviation 0.005 20.5 / 21.5 / 30.2, with
// such keys too 21.8 / 25.6 / 39.4 (key by key in fp32, as only values that are not finite go,
// 104 / 184 / 344).
//
// Softmax: running maximum and sum per row in fp32, in the log2 domain.  On a bf16 cache a
// weight p goes to the second product as bf16(p) + bf16(p - bf16(p)), 16 significant bits:
// one bf16 alone would add an error as large as the output's own rounding (2^-9 per weight).
// Over fp16 values one fp16 weight has 11 bits, and a second product is not needed.
//
// The list is cut into up to 8 slices, one CTA of a thread-block cluster each; the parts are
// joined through distributed shared memory in a fixed order, so a call is one launch, needs
// no workspace and repeats bit for bit.
//
// Measured, d = 128: 16 sequences of 16384 rows, 32 query heads on 8, one token, e4m3, lists
// of about 4400 keys: 44 us, 3.4 TB/s of codes and scales gathered, 52 % of the card's copy
// rate.  DRAM runs at 41 % of its peak and the schedulers issue in 39 % of the cycles: with 128
// registers a thread an SM holds 16 of these warps, which wait in turn for their gathers
// (stalls 1.2 an issued instruction), for their own arithmetic (1.5) and for shared memory
// (0.7); and 512 CTAs leave 14 % of the places for 592 empty.  One sequence, bf16, 1-token
// step: 8.8 us, a chain of a launch, the lists, the look-ups, a gather and the join.
#include <atomic>
#include <type_traits>

#include "trace.h"
#include "tree.cuh"

namespace ssa {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_half(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a CTA works out once, and each warp's resolved entries: two batches of 32.
template <int ROWS>
struct Shared : TreeInfo {
    int key[kWarps * 64];          // cache row
    uint32_t mask[kWarps * 64];    // bit i: row i retains the key
    uint32_t here;                 // the first 16 heads
    uint32_t spread[4][16];        // rows of four heads' bits
    uint32_t node_rows[64];        // rows that retain a node
    Problem w;
    const uint16_t *q_rows[ROWS];  // Q's row, or null behind the last
};

// Row bits of an entry: bit i = row i retains the key.  An entry that no row retains
// gets no bits and the first node's row, which is there to be read.
template <int ROWS>
__device__ __forceinline__ void resolve(const Entry &x, const TreeParams &p, const Problem &w, const Shared<ROWS> &sh,
                                        int &key, uint32_t &bits) {
    int j, o, node;
    uint32_t marks;
    x.place(w, j, o, node, marks);
    RowBits<1> row_bits{};
    uint32_t &rows = row_bits.v[0];
    if (j < 0) {
    } else if (node >= 0) {
        rows = sh.node_rows[node];
    } else {
        rows = sh.spread[0][marks & 15];
        if (w.G > 4)
            rows |= sh.spread[1][(marks >> 4) & 15] | sh.spread[2][(marks >> 8) & 15] | sh.spread[3][(marks >> 12) & 15];
        row_bits.look_up_heads(p, w, sh, (marks >> 16) & ~marks & sh.here, j, o);
    }
    bits = rows;
    key = rows ? j : w.len;
}

// ---------------------------------------------------------------------------------
// A warp's share of the keys
// ---------------------------------------------------------------------------------
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that the 16-high
// operand is the cache and NT blocks of 8 rows are the narrow one.  Each warp takes 16 keys
// at a time on its own.  A product's inner index may be permuted, so lane (q, n) =
// (lane & 3, lane >> 2) supplies for the keys n and n + 8 of the first product the D/4
// consecutive elements from q D/4 on, and for the second, whose inner index is the key, the
// D/8 elements from n D/8 on of the keys 2q, 2q + 1, 2q + 8, 2q + 9: wide loads of whole
// rows, one scale group a lane, no shared memory.  The transposed weights become the second
// product's operand by an 8x8 transpose within the warp (movmatrix); a lane ends up with D/8
// consecutive outputs of the rows 2q and 2q + 1 of each block, and its logits are of the
// same rows, so rescaling O needs no exchange either.
//
// The reference of the softmax moves only when a logit exceeds it by 2^8, less kLift (weights
// then stay below 2^15, sums in fp32): one vote a step instead of a maximum over the warp.
//
// Rows travel by cp.async into a ring of three steps of the warp's own, two steps ahead of
// their use: 2 x 4 KB a warp in flight (e4m3, d = 128) without a register, no CTA barrier.
// The 16-byte pieces of a row are permuted by the row's number so that both products' loads
// are free of bank conflicts.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t *w) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr)
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}

// The ring: a step holds 16 key rows, then 16 value rows.
template <int D, int FMT>
struct Ring {
    static constexpr int kRow = kv_row_bytes(FMT, D), kPieces = kRow / 16;  // 2, 4, 8 or 16 of 16 bytes
    static constexpr int kStep = 32 * kRow, kSteps = 3, kBytes = kSteps * kStep;
    // A lane's share of a key row: pieces [q, 4 + q, ..] of a 256-byte row, else a quarter of
    // it in one run; of a value row an eighth in one run.
    static constexpr int kKeyWords = kRow / 16, kValWords = kRow / 32;

    static __device__ __forceinline__ uint32_t swizzle(uint32_t row) {
        if constexpr (kPieces == 16) return ((row >> 1) & 1) | ((((row >> 2) ^ row) & 1) << 2);
        else if constexpr (kPieces == 8) return row & 7;
        else if constexpr (kPieces == 4) return (row >> 1) & 3;
        else return (row >> 2) & 1;
    }
    static __device__ __forceinline__ uint32_t piece(uint32_t base, uint32_t row, uint32_t c) {
        return base + row * kRow + ((c ^ swizzle(row)) << 4);
    }
    // first word of a lane's part (bytes, a multiple of 4) within a row
    static __device__ __forceinline__ uint32_t word(uint32_t base, uint32_t row, uint32_t bytes) {
        return piece(base, row, bytes >> 4) + (bytes & 15);
    }
    static __device__ __forceinline__ void load_key(uint32_t base, uint32_t row, uint32_t q, uint32_t *w) {
        if constexpr (kPieces == 16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) lds_words<4>(piece(base, row, q + 4 * j), w + 4 * j);
        } else if constexpr (kKeyWords >= 4) {
#pragma unroll
            for (int j = 0; j < kKeyWords / 4; ++j) lds_words<4>(piece(base, row, q * (kKeyWords / 4) + j), w + 4 * j);
        } else {
            lds_words<kKeyWords>(word(base, row, q * kKeyWords * 4), w);
        }
    }
    static __device__ __forceinline__ void load_val(uint32_t base, uint32_t row, uint32_t n, uint32_t *w) {
        if constexpr (kValWords >= 4) {
#pragma unroll
            for (int j = 0; j < kValWords / 4; ++j) lds_words<4>(piece(base, row, n * (kValWords / 4) + j), w + 4 * j);
        } else {
            lds_words<kValWords>(word(base, row, n * kValWords * 4), w);
        }
    }
    // element of a query row that a lane's i-th key word pair starts at (bf16 words of Q)
    static __device__ __forceinline__ int query_at(int q, int piece8) {  // the lane's piece of 8 elements
        return kPieces == 16 ? 8 * (q + 4 * piece8) : q * (D / 4) + 8 * piece8;
    }
};

template <int D, int FMT, int NT>
struct Warp {
    using R = Ring<D, FMT>;
    using VRun = Run<FMT, D / 8>;
    static constexpr bool kHalf = FMT != SSA_KV_BF16;
    static constexpr bool kQueryShared = NT > 2;  // O takes the registers; the CTA's fragments lie in shared memory
    static constexpr int kQueryBytes = kQueryShared ? NT * (D / 16) * 32 * 8 : 0;

    uint32_t qb[kQueryShared ? 1 : NT][D / 16][2];
    uint32_t q_smem;           // this lane's fragment (t, s) is at q_smem + 256 (t D/16 + s)
    float scale[NT][2];       // of the rows 2q, 2q + 1: logit in the log2 domain per unit of product
    float o[NT][D / 16][4];   // tile j: elements 2j, 2j + 1 of the lane's run x rows 2q, 2q + 1
    float m[NT][2], l[NT][2];  // reference (log2 domain), this lane's sum
    uint32_t sc[3];            // scale bytes of row lane % 16 of the keys (lanes 0-15) or values, by step

    __device__ __forceinline__ void init() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[t][j][c] = 0.0f;
            m[t][0] = m[t][1] = -3.402823466e38f;  // finite: differences with it are never NaN
            l[t][0] = l[t][1] = 0.0f;
        }
    }

    // src[t]: row 8t + n of the block, or null
    static __device__ __forceinline__ void fetch_q(const uint16_t *const (&src)[NT], uint32_t (&words)[NT][D / 8]) {
        const int q = threadIdx.x & 3;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t x[4] = {0, 0, 0, 0};
                if (src[t]) load_words<4>(reinterpret_cast<const uint8_t *>(src[t] + R::query_at(q, i)), x);
#pragma unroll
                for (int u = 0; u < 4; ++u) words[t][4 * i + u] = x[u];
            }
        }
    }
    // For fp16 products a row is scaled (query_shift).
    __device__ __forceinline__ void set_q(uint32_t (&words)[NT][D / 8], float scale_log2, uint8_t *shared) {
        const int lane = threadIdx.x & 31, q = lane & 3;
        q_smem = smem_u32(shared) + 8 * lane;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t (&w)[D / 8] = words[t];
            scale[t][0] = scale[t][1] = scale_log2;
            if constexpr (kHalf) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
                    top = max(top, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int up = query_shift(top);
                const float f = power_of_two(up);
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    w[i] = pack_half(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
                const float down = shifted_scale(scale_log2, up);
#pragma unroll
                for (int k = 0; k < 2; ++k) scale[t][k] = __shfl_sync(0xffffffffu, down, (2 * q + k) * 4);
            }
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                if constexpr (kQueryShared) {
                    if (threadIdx.x < 32)
                        *reinterpret_cast<uint2 *>(shared + 8 * lane + 256 * (t * (D / 16) + s)) =
                            make_uint2(w[2 * s], w[2 * s + 1]);
                } else {
                    qb[t][s][0] = w[2 * s];
                    qb[t][s][1] = w[2 * s + 1];
                }
            }
        }
    }

    // Starts the copies of a step's 16 keys and values, and loads their scales.
    __device__ __forceinline__ void issue(const Rows &rows, const int *key, uint32_t dst, uint32_t &scales) {
        const int lane = threadIdx.x & 31;
        constexpr int kPer = 32 / R::kPieces;  // rows a warp copies at a time
        const uint32_t c = lane % R::kPieces;
#pragma unroll
        for (int i = 0; i < 16 / kPer; ++i) {
            const uint32_t r = i * kPer + lane / R::kPieces;
            const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(key[r])) * R::kRow + 16 * c;
            copy16(R::piece(dst, r, c), rows.k + at);
            copy16(R::piece(dst + 16 * R::kRow, r, c), rows.v + at);
        }
        if constexpr (kHalf) {
            const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(key[lane & 15])) * (D / SSA_KV_GROUP);
            const uint8_t *src = (lane < 16 ? rows.ks : rows.vs) + at;
            if constexpr (D == 128) scales = __ldg(reinterpret_cast<const uint32_t *>(src));
            else scales = __ldg(reinterpret_cast<const uint16_t *>(src));
        }
    }

    // Weights of the step's 16 keys from its logits; x[t]: {key n, n + 8} x {rows 2q, 2q + 1}
    __device__ __forceinline__ void weights(float (&x)[NT][4], uint32_t mask0, uint32_t mask1) {
        const int lane = threadIdx.x & 31, q = lane & 3;
        float y[NT][4];
        bool over = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool in = (((c & 2) ? mask1 : mask0) >> (8 * t + 2 * q + (c & 1))) & 1;
                if (!in) x[t][c] = -INFINITY;
                y[t][c] = fmaf(x[t][c], scale[t][c & 1], -m[t][c & 1]);
                over |= y[t][c] > kSlack + kLift<kHalf>;
            }
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float top = fmaxf(m[t][k], fmaf(fmaxf(x[t][k], x[t][2 + k]), scale[t][k], -kLift<kHalf>));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const float f = ex2_approx(m[t][k] - top);
                    if (m[t][k] != top) {  // not inf - inf
                        l[t][k] *= f;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            o[t][j][k] *= f;
                            o[t][j][2 + k] *= f;
                        }
                    }
                    m[t][k] = top;
                    y[t][k] = fmaf(x[t][k], scale[t][k], -top);
                    y[t][2 + k] = fmaf(x[t][2 + k], scale[t][k], -top);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // a key that the row does not retain has no weight, whatever the reference
                x[t][c] = x[t][c] == -INFINITY ? 0.0f : ex2_approx(y[t][c]);
                l[t][c & 1] += x[t][c];
            }
        }
    }

    // One step: the 16 keys of a ring step.
    __device__ __forceinline__ void step(const Rows &rows, const uint16_t *const *q_rows, const int *key,
                                         const uint32_t *mask, uint32_t base, uint32_t scales, float scale_log2,
                                         int32_t *status) {
        const int lane = threadIdx.x & 31, q = lane & 3, n = lane >> 2;
        uint32_t plain = 0xffffffffu;  // rows (keys, then values) whose scales are all exact in fp16
        if constexpr (kHalf) {
            uint32_t worst = 0;
#pragma unroll
            for (int i = 0; i < D / SSA_KV_GROUP; ++i) worst = max(worst, ((scales >> (8 * i)) & 255u) - kScaleHalf);
            plain = __ballot_sync(0xffffffffu, worst <= kv_scale_max(FMT) - kScaleHalf);
        }
        float x[NT][4] = {};
        if ((plain & 0xffffu) != 0xffffu) {
            logits_of_small_keys(q_rows, base, scales, scale_log2, x);
        } else {
            uint32_t kw[2][R::kKeyWords];
            R::load_key(base, n, q, kw[0]);
            R::load_key(base, n + 8, q, kw[1]);
            uint32_t f[2] = {0, 0};
            if constexpr (kHalf) {
                const int group = 8 * (q * (D / 4) / SSA_KV_GROUP);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t E = (__shfl_sync(0xffffffffu, scales, n + 8 * k) >> group) & 255u;
                    f[k] = half_factors(E, E);
                }
            }
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                uint32_t a[4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if constexpr (FMT == SSA_KV_E4M3) {
                        a[k] = h2_mul(half_e4m3(kw[k][s]), f[k]);
                        a[2 + k] = h2_mul(half_e4m3(kw[k][s] >> 16), f[k]);
                    } else if constexpr (FMT == SSA_KV_E2M1) {
                        uint32_t h[4];
                        half_e2m1(kw[k][s / 2], h);
                        a[k] = h2_mul(h[2 * (s & 1)], f[k]);
                        a[2 + k] = h2_mul(h[2 * (s & 1) + 1], f[k]);
                    } else {
                        a[k] = kw[k][2 * s];
                        a[2 + k] = kw[k][2 * s + 1];
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    uint32_t b[2];
                    if constexpr (kQueryShared) {
                        lds_words<2>(q_smem + 256 * (t * (D / 16) + s), b);
                    } else {
                        b[0] = qb[t][s][0];
                        b[1] = qb[t][s][1];
                    }
                    if constexpr (kHalf) mma_half(x[t], a, b[0], b[1]);
                    else mma_bf16(x[t], a, b[0], b[1]);
                }
            }
        }
        weights(x, mask[n], mask[8 + n]);
        uint32_t vw[4][R::kValWords];
#pragma unroll
        for (int t = 0; t < 4; ++t) R::load_val(base + 16 * R::kRow, 2 * q + (t & 1) + 8 * (t >> 1), n, vw[t]);
        bool odd = false, small = false;  // values that are not finite; values for bf16
        if constexpr (kHalf) {
            if (plain != 0xffffffffu) {
                bool big = false;
#pragma unroll
                for (int i = 0; i < D / SSA_KV_GROUP; ++i) {
                    const uint32_t E = (scales >> (8 * i)) & 255u;
                    big |= E > kv_scale_max(FMT);
                    if (kv_bad_scale(FMT, E)) report(status, SSA_ERR_INVALID);
                }
                odd = (__ballot_sync(0xffffffffu, big) >> 16) != 0;
                small = !odd && (plain >> 16) != 0xffffu;
            }
        } else {
            uint32_t c = 0;  // x * 0 is NaN for an infinity or a NaN, and stays one
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < R::kValWords; ++i) c = bf2_fma(vw[t][i], 0u, c);
            odd = __any_sync(0xffffffffu, (c & 0x7fff7fffu) != 0);
        }
        if (odd) {
            one_by_one(rows, key, mask, x);
        } else if (!kHalf || small) {
            products_bf16(base, scales, vw, x);
        } else if constexpr (kHalf) {
            // weights as fp16: 2^-12 of the weight, or 2^-25 where it is below 2^-14 (the largest
            // is 2^7 or more): against the output's 2^-9 one product is enough
            uint32_t w[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int k = 0; k < 2; ++k) w[t][k] = transpose8x8(pack_half(x[t][2 * k], x[t][2 * k + 1]));
            }
            uint32_t E[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                E[t] = (__shfl_sync(0xffffffffu, scales, 16 + 2 * q + (t & 1) + 8 * (t >> 1)) >>
                        (8 * (n * (D / 8) / SSA_KV_GROUP))) & 255u;
            const uint32_t f01 = half_factors(E[0], E[1]), f23 = half_factors(E[2], E[3]);
            // the codes of two keys are paired before they are converted
            const auto product = [&](int j, const uint32_t(&c)[4]) {
                const uint32_t a[4] = {h2_mul(c[0], f01), h2_mul(c[1], f01), h2_mul(c[2], f23), h2_mul(c[3], f23)};
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_half(o[t][j], a, w[t][0], w[t][1]);
            };
            if constexpr (FMT == SSA_KV_E4M3) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {  // elements 2j, 2j + 1
                    const uint32_t s0 = (j & 1) ? 0x62u : 0x40u, s1 = (j & 1) ? 0x73u : 0x51u;
                    const uint32_t c[4] = {half_e4m3(prmt(vw[0][j / 2], vw[1][j / 2], s0)),
                                           half_e4m3(prmt(vw[0][j / 2], vw[1][j / 2], s1)),
                                           half_e4m3(prmt(vw[2][j / 2], vw[3][j / 2], s0)),
                                           half_e4m3(prmt(vw[2][j / 2], vw[3][j / 2], s1))};
                    product(j, c);
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {  // a word of 8 elements of each key
                    uint32_t even[2][4], odds[2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t a = vw[2 * k][i], b = vw[2 * k + 1][i];
                        half_e2m1((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), even[k]);
                        half_e2m1(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), odds[k]);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t c[4] = {even[0][u], odds[0][u], even[1][u], odds[1][u]};
                        product(4 * i + u, c);
                    }
                }
            }
        }
    }

    // The scale bytes of a row from lane `src`, and the factor of its group `g`.
    static __device__ __forceinline__ uint32_t row_factor(uint32_t scales, int src, int g) {
        return kv_factor<FMT>((__shfl_sync(0xffffffffu, scales, src) >> (8 * g)) & 255u);
    }

    // Logits where a scale is below fp16's exact range: the step's keys as bf16, with Q's rows as
    // they are.
    __device__ __forceinline__ void logits_of_small_keys(const uint16_t *const *q_rows, uint32_t base, uint32_t scales,
                                                         float scale_log2, float (&x)[NT][4]) const {
        if constexpr (kHalf) {
            const int lane = threadIdx.x & 31, q = lane & 3, n = lane >> 2;
            uint32_t f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) f[k] = row_factor(scales, n + 8 * k, q * (D / 4) / SSA_KV_GROUP);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t kw[2][R::kKeyWords];
                R::load_key(base, n, q, kw[0]);
                R::load_key(base, n + 8, q, kw[1]);
                const uint16_t *const src[1] = {q_rows[8 * t + n]};
                uint32_t w[1][D / 8];
                Warp<D, FMT, 1>::fetch_q(src, w);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    uint32_t a[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t u, v;
                        if constexpr (FMT == SSA_KV_E4M3) {
                            decode_e4m3(kw[k][s], f[k], u, v);
                            a[k] = prmt(u, v, 0x5410u);
                            a[2 + k] = prmt(u, v, 0x7632u);
                        } else {
                            decode_e2m1(kw[k][s / 2] >> (16 * (s & 1)), f[k], a[k], a[2 + k]);
                        }
                    }
                    mma_bf16(x[t], a, w[0][2 * s], w[0][2 * s + 1]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) x[t][c] *= scale_log2 / scale[t][c & 1];  // in the units of the row's products
            }
        }
    }

    // O += V^T P^T over bf16 values, those of a bf16 cache or decoded, with P in two parts.
    __device__ __forceinline__ void products_bf16(uint32_t base, uint32_t scales, const uint32_t (&vw)[4][R::kValWords],
                                                  const float (&x)[NT][4]) {
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float a = x[t][2 * k], b = x[t][2 * k + 1];
                const uint32_t w = pack_bf16(a, b);
                hi[t][k] = transpose8x8(w);
                lo[t][k] = transpose8x8(pack_bf16(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xffff0000u)));
            }
        }
        const auto product = [&](int j, const uint32_t(&a)[4]) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mma_bf16(o[t][j], a, hi[t][0], hi[t][1]);
                mma_bf16(o[t][j], a, lo[t][0], lo[t][1]);
            }
        };
        if constexpr (!kHalf) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t a[4] = {prmt(vw[0][j], vw[1][j], 0x5410u), prmt(vw[0][j], vw[1][j], 0x7632u),
                                       prmt(vw[2][j], vw[3][j], 0x5410u), prmt(vw[2][j], vw[3][j], 0x7632u)};
                product(j, a);
            }
        } else {
            const int lane = threadIdx.x & 31, q = lane & 3, n = lane >> 2;
            uint32_t f[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                f[t] = row_factor(scales, 16 + 2 * q + (t & 1) + 8 * (t >> 1), n * (D / 8) / SSA_KV_GROUP);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {  // four elements of each key
                uint32_t u[4], v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {  // read again: held since the fast path's load, the words would be spilled
                    uint32_t w;
                    lds_words<1>(R::word(base + 16 * R::kRow, 2 * q + (t & 1) + 8 * (t >> 1),
                                         4 * (n * R::kValWords + (FMT == SSA_KV_E4M3 ? i : i / 2))),
                                 &w);
                    if constexpr (FMT == SSA_KV_E4M3) decode_e4m3(w, f[t], u[t], v[t]);
                    else decode_e2m1(w >> (16 * (i & 1)), f[t], u[t], v[t]);
                }
                if constexpr (FMT == SSA_KV_E4M3) {  // u: elements 0 and 2, v: 1 and 3
                    const uint32_t a[4] = {prmt(u[0], u[1], 0x5410u), prmt(v[0], v[1], 0x5410u), prmt(u[2], u[3], 0x5410u),
                                           prmt(v[2], v[3], 0x5410u)};
                    const uint32_t b[4] = {prmt(u[0], u[1], 0x7632u), prmt(v[0], v[1], 0x7632u), prmt(u[2], u[3], 0x7632u),
                                           prmt(v[2], v[3], 0x7632u)};
                    product(2 * i, a);
                    product(2 * i + 1, b);
                } else {  // u: elements 0 and 1, v: 2 and 3
                    const uint32_t a[4] = {prmt(u[0], u[1], 0x5410u), prmt(u[0], u[1], 0x7632u), prmt(u[2], u[3], 0x5410u),
                                           prmt(u[2], u[3], 0x7632u)};
                    const uint32_t b[4] = {prmt(v[0], v[1], 0x5410u), prmt(v[0], v[1], 0x7632u), prmt(v[2], v[3], 0x5410u),
                                           prmt(v[2], v[3], 0x7632u)};
                    product(2 * i, a);
                    product(2 * i + 1, b);
                }
            }
        }
    }

    // Values that are not finite: 0 * infinity would reach rows that do not retain the key,
    // and the remainder's sign rows that do.  Key by key, only where the row's bit is set.
    __device__ __forceinline__ void one_by_one(const Rows &rows, const int *key, const uint32_t *mask,
                                               const float (&x)[NT][4]) {
        const int lane = threadIdx.x & 31, q = lane & 3, n = lane >> 2;
#pragma unroll 1
        for (int kk = 0; kk < 16; ++kk) {
            const int src = (kk & 7) * 4 + q;
            float w[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                w[t][0] = __shfl_sync(0xffffffffu, kk < 8 ? x[t][0] : x[t][2], src);
                w[t][1] = __shfl_sync(0xffffffffu, kk < 8 ? x[t][1] : x[t][3], src);
            }
            VRun run;
            run.load(rows.v, rows.vs, key[kk], D, n);
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
                const float v = run.value(e);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float &acc = o[t][e / 2][2 * (e & 1) + k];
                        if ((mask[kk] >> (8 * t + 2 * q + k)) & 1) acc = fmaf(w[t][k], v, acc);
                    }
                }
            }
        }
        __syncwarp();  // key and mask are read: the next batch may take their place
    }

    // The list in batches of 32 entries, dealt out to the warps of all slices in turn (the
    // costlier entries, columns, lie together at its end).  An entry is fetched three batches
    // ahead, probed two and resolved one ahead; the first two come fetched, the first probed.
    template <int ROWS>
    __device__ __forceinline__ void run(const TreeParams &p, const Problem &w, Shared<ROWS> &sh, const Rows &rows,
                                        int total, int e0, Entry now, Entry next, uint32_t ring) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int stride = 32 * kWarps * p.slices;
        int *key = sh.key + warp * 64;
        uint32_t *mask = sh.mask + warp * 64;
        int at = e0 + lane;
        const auto resolve = [&](const Entry &x, int slot) {
            uint32_t bits;
            int j;
            ssa::resolve<ROWS>(x, p, w, sh, j, bits);
            key[slot + lane] = j;
            mask[slot + lane] = bits;
        };
        if (e0 >= total) return;
        resolve(now, 0);
        __syncwarp();
        issue(rows, key, ring, sc[0]);
        asm volatile("cp.async.commit_group;" ::: "memory");
        issue(rows, key + 16, ring + R::kStep, sc[1]);
        asm volatile("cp.async.commit_group;" ::: "memory");
        now = next;
        now.probe(w);
        next.fetch(w, at + 2 * stride);
        int slot = 0;
        uint32_t here = 0, ahead = 2 * R::kStep;  // ring steps: the one in use, the one to fill
        for (; e0 < total; e0 += stride) {
            const bool more = e0 + stride < total;
            if (more) {
                resolve(now, slot ^ 32);
                now = next;
                now.probe(w);
                at += stride;
                next.fetch(w, at + 2 * stride);
            }
#pragma unroll 1
            for (int i = 0; i < 32; i += 16) {
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncwarp();  // all lanes' copies of this step are there, and the step to fill is free
                if (more) issue(rows, key + (slot ^ 32) + i, ring + ahead, sc[2]);
                asm volatile("cp.async.commit_group;" ::: "memory");
                step(rows, sh.q_rows, key + slot + i, mask + slot + i, ring + here, sc[0], p.scale_log2, p.status);
                sc[0] = sc[1];
                sc[1] = sc[2];
                here = here == 2 * R::kStep ? 0 : here + R::kStep;
                ahead = ahead == 2 * R::kStep ? 0 : ahead + R::kStep;
            }
            slot ^= 32;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();  // the ring is free for the warp's part
    }

    // O, the references and the sums of the block's rows to a part in shared memory
    __device__ __forceinline__ void store(float *part, int pitch, float (*ml)[2]) {
        const int lane = threadIdx.x & 31, q = lane & 3, n = lane >> 2;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = 8 * t + 2 * q + k;
                float e[D / 8];
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int u = 0; u < 4; ++u) e[4 * j + u] = o[t][2 * j + (u >> 1)][2 * (u & 1) + k];
#pragma unroll
                for (int i = 0; i < D / 8; i += 4)
                    *reinterpret_cast<float4 *>(part + row * pitch + n * (D / 8) + i) =
                        make_float4(e[i], e[i + 1], e[i + 2], e[i + 3]);
                float sum = l[t][k];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (n == 0) {
                    ml[row][0] = m[t][k];
                    ml[row][1] = sum;
                }
            }
        }
    }
};

template <int D, int FMT, int ROWS>
struct Layout {
    static constexpr int kPartPitch = D + 4;  // floats
    static constexpr int kPart = ROWS * kPartPitch * 4;
    // a warp's ring, later its part; behind the rings the query fragments
    static constexpr int kWarpBytes = Ring<D, FMT>::kBytes > kPart ? Ring<D, FMT>::kBytes : kPart;
    static constexpr int kBytes = kWarps * kWarpBytes + Warp<D, FMT, ROWS / 8>::kQueryBytes;
};

// CTAs that run at once on an SM (registers; shared memory for the larger rings).
constexpr int resident_ctas(int d, int fmt, int rows) {
    if (rows == 8) return d == 64 ? (fmt == SSA_KV_BF16 ? 4 : 5) : fmt == SSA_KV_BF16 ? 2 : 4;
    if (rows == 16) return d == 64 ? 3 : 2;
    return 2;
}

// ---------------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------------

template <int D, int FMT, int ROWS>
__global__ void __launch_bounds__(32 * kWarps, resident_ctas(D, FMT, ROWS)) attn_tree_kernel(const TreeParams p) {
    using L = Layout<D, FMT, ROWS>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Shared<ROWS> sh;
    __shared__ float s_ml[kWarps][ROWS][2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slice = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    cg::cluster_group cluster = cg::this_cluster();

    const int len = __ldg(p.len + b);
    int nn = p.nodes ? __ldg(p.nodes + b) : p.T;
    const int hp = __ldg(p.head_ptr + g), G = __ldg(p.head_ptr + g + 1) - hp;
    bool bad = len < 0 || nn < 0 || nn > p.T || static_cast<long long>(len) + nn > p.S;
    nn = min(max(nn, 0), p.T);
    const int last = min(ROWS, G * nn);  // rows
    if (last == 0) {                     // every CTA of the cluster alike
        if (bad && g == 0 && slice == 0 && tid == 0) report(p.status, SSA_ERR_INVALID);
        return;
    }
    if (tid == 0) {
        sh.bad = bad;
        sh.max_depth = 0;
        set_problem(p, sh.w, g, len, nn, 0, last, hp, G);
        sh.here = (1u << min(G, 16)) - 1;
    } else if (tid == 32) {
        set_lengths(p, sh.w, g, len, bad);
    } else if (tid >= 64) {
        const int set = (tid - 64) >> 4;
        uint32_t rows = 0;
        for (int k = 0; k < 4; ++k) {
            const int lo = (4 * set + k) * nn, hi = min(lo + nn, last);
            if (((tid >> k) & 1) && lo < hi) rows |= (0xffffffffu >> (32 - (hi - lo))) << lo;
        }
        sh.spread[set][tid & 15] = rows;
        if (set == 3) set_heads(p, sh.w, hp, G, tid & 15);
    }
    __syncthreads();
    const Problem &w = sh.w;
    Warp<D, FMT, ROWS / 8> acc;
    // what needs no more than the lengths of the lists is loaded while the tree is worked out
    const uint16_t *src[ROWS / 8];
#pragma unroll
    for (int k = 0; k < ROWS / 8; ++k) {
        const int r = (lane >> 2) + 8 * k;
        src[k] = r < last ? p.Q + row_index(p, w, b, r) * D : nullptr;
        if ((lane & 3) == 0 && warp == 0) sh.q_rows[(lane >> 2) + 8 * k] = src[k];
    }
    uint32_t q_words[ROWS / 8][D / 8];
    acc.fetch_q(src, q_words);
    const int e0 = 32 * (slice * kWarps + warp);
    Entry now, next;
    now.fetch(w, e0 + lane);
    next.fetch(w, e0 + lane + 32 * kWarps * p.slices);
    now.probe(w);
    resolve_tree(p, sh, b, nn);
    __syncthreads();
    if (warp == 3) transpose_nodes(lane < last && !bad ? retained_nodes(p, w, sh, lane) : 0, nn, sh.node_rows);
    acc.set_q(q_words, p.scale_log2, smem + kWarps * L::kWarpBytes);
    acc.init();
    __syncthreads();
    bad = sh.bad;
    if (bad && slice == 0 && tid == 0) report(p.status, SSA_ERR_INVALID);

    const Rows rows = rows_of<D, FMT>(p, b, g);
    acc.template run<ROWS>(p, w, sh, rows, bad ? 0 : w.n_off + w.n_col + nn, e0, now, next,
                           smem_u32(smem) + warp * L::kWarpBytes);

    // parts: per warp O, the references and the sums
    float *parts = reinterpret_cast<float *>(smem);
    acc.store(parts + warp * (L::kWarpBytes / 4), L::kPartPitch, s_ml[warp]);
    if (p.slices > 1) cluster.sync();
    else __syncthreads();

    join_parts<D, kWarps>(
        p, w, b, slice, warp, kWarps, [&](int c, int i) { return s_ml[c][i]; },
        [&](int c, int i) { return parts + c * (L::kWarpBytes / 4) + i * L::kPartPitch; });
    if (p.slices > 1) cluster.sync();  // a part stays until the cluster has read it
}

template <int D, int FMT, int ROWS>
int launch_tree(TreeParams &p, int entries, cudaStream_t s) {
    using L = Layout<D, FMT, ROWS>;
    auto kernel = attn_tree_kernel<D, FMT, ROWS>;
    int device = 0;
    SSA_CUDA_TRY(cudaGetDevice(&device));
    if (L::kBytes > 40 * 1024) {  // once per device
        static std::atomic<uint64_t> done{0};
        const uint64_t bit = device < 64 ? 1ull << device : 0;
        if (!(done.load() & bit)) {
            SSA_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes));
            done.fetch_or(bit);
        }
    }
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = L::kBytes;
    // Slices of the list: as many as run at once, with 64 keys each at least.  16 sequences x 8 KV
    // heads over 4400 e4m3 keys: 4 slices 44 us, 5, 6 and 8 slices (a second wave) 65, 59 and 57.
    static ClusterCounts clusters;
    p.slices = pick_slices(kernel, cfg, clusters, device, static_cast<long long>(p.B) * p.Hkv, entries / 64);
    cfg.gridDim = dim3(p.slices, p.Hkv, p.B);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.slices;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.slices > 1 ? 1 : 0;
    SSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
    return SSA_OK;
}

// The fewest blocks of 8 rows that hold them: 16 sequences over lists of 5000 e4m3 keys took
// 50 us with 8 rows a CTA where the 32-row kernel took 85, and 70 us with 16 where it took 88.
template <int D, int FMT>
int launch_rows(TreeParams &p, int rows, int entries, cudaStream_t s) {
    if (rows <= 8) return launch_tree<D, FMT, 8>(p, entries, s);
    if (rows <= 16) return launch_tree<D, FMT, 16>(p, entries, s);
    return launch_tree<D, FMT, 32>(p, entries, s);
}

template <int D>
int launch_format(TreeParams &p, int fmt, int rows, int entries, cudaStream_t s) {
    if (fmt == SSA_KV_BF16) return launch_rows<D, SSA_KV_BF16>(p, rows, entries, s);
    if (fmt == SSA_KV_E4M3) return launch_rows<D, SSA_KV_E4M3>(p, rows, entries, s);
    return launch_rows<D, SSA_KV_E2M1>(p, rows, entries, s);
}

}  // namespace
}  // namespace ssa

using namespace ssa;

extern "C" int sparse_attn_tree(const void *Q, const ssa_kv_cache *cache, int H_q, int T, const int32_t *len,
                                const int32_t *n_nodes, const int32_t *parent, const ssa_tree_lists *lists, float scale,
                                void *O, float *LSE, int32_t *dev_status, void *stream) {
    ssa::TraceRange trace_range("sparse_attn_tree");
    if (const int rc = check_cache("sparse_attn_tree", cache)) return rc;
    SSA_CHECK_ARG(Q && len && lists && O && LSE, "sparse_attn_tree: null pointer argument");
    SSA_CHECK_ARG(T >= 1 && T <= SSA_TREE_MAX, "sparse_attn_tree: T must be in [1, %d]", SSA_TREE_MAX);
    const ssa_tree_sizes &z = lists->sizes;
    SSA_CHECK_ARG(z.n_heads == H_q && z.H_kv == cache->H_kv && z.S == cache->S,
                  "sparse_attn_tree: lists (S=%d heads=%d/%d) do not match S=%d H_q=%d H_kv=%d", z.S, z.n_heads, z.H_kv,
                  cache->S, H_q, cache->H_kv);
    SSA_CHECK_ARG(z.depth >= 1 && z.depth <= SSA_TREE_MAX && z.words == z.S / 64 + 2 && z.max_group >= 1 &&
                      z.max_group <= z.n_heads && z.max_entries >= 0,
                  "sparse_attn_tree: the lists' sizes are not those of sparse_tree_lists");
    SSA_CHECK_ARG(lists->diag_bits && lists->col_bits && lists->group_offs && lists->group_cols && lists->off_rank &&
                      lists->col_rank && lists->off_ptr && lists->offs && lists->col_ptr && lists->cols &&
                      lists->head_ptr && lists->heads,
                  "sparse_attn_tree: null list buffer");
    SSA_CHECK_ARG(aligned16(lists->offs) && aligned16(lists->cols),
                  "sparse_attn_tree: offs and cols must be 16-byte aligned");
    SSA_CHECK_ARG(aligned16(Q) && aligned16(O) && Q != O, "sparse_attn_tree: Q and O must be 16-byte aligned and distinct");
    SSA_CHECK_ARG(scale > 0.0f && scale < 1e30f, "sparse_attn_tree: scale must be positive and finite");
    SSA_CHECK_ARG(static_cast<long long>(z.max_group) * T <= (1 << 20), "sparse_attn_tree: too many rows per KV head");
    TreeParams p{};
    p.B = cache->B;
    p.T = T;
    p.H = H_q;
    p.Hkv = cache->H_kv;
    p.S = cache->S;
    p.depth = z.depth;
    p.words = z.words;
    p.Q = static_cast<const uint16_t *>(Q);
    p.ck = static_cast<const uint8_t *>(cache->k);
    p.cv = static_cast<const uint8_t *>(cache->v);
    p.sk = cache->k_scale;
    p.sv = cache->v_scale;
    p.len = len;
    p.nodes = n_nodes;
    p.parent = parent;
    p.dbits = lists->diag_bits;
    p.cbits = lists->col_bits;
    p.goffs = lists->group_offs;
    p.gcols = lists->group_cols;
    p.off_rank = lists->off_rank;
    p.col_rank = lists->col_rank;
    p.off_ptr = lists->off_ptr;
    p.offs = lists->offs;
    p.col_ptr = lists->col_ptr;
    p.cols = lists->cols;
    p.head_ptr = lists->head_ptr;
    p.heads = lists->heads;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.O = static_cast<uint16_t *>(O);
    p.LSE = LSE;
    p.status = dev_status;
    p.wait_ns = wait_limit_ns();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int rows = z.max_group * T, entries = z.max_entries + T;
    // Up to 32 rows here, more on 128-row tiles in tensor memory, whose time hardly depends on
    // the rows.  16 sequences over lists of 7400 / 900 e4m3 keys: 32 rows 122 / 25.8 us here,
    // 165 / 26.5 there; 36 rows, two blocks of 32, 221 / 37.3 here, 172 / 28.0 there (bf16: 139
    // and 182 us, 266 and 192 us).
    if (rows > 32) return launch_tree_wide(p, cache->d, cache->format, rows, entries, s);
    return cache->d == 64 ? launch_format<64>(p, cache->format, rows, entries, s)
                          : launch_format<128>(p, cache->format, rows, entries, s);
}
