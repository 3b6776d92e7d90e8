// tree.cuh -- what the kernels of the tree attention share: the list entries of a problem and
// the rows that retain them, decoding of cache rows, joining the parts of a cluster.
#pragma once

#include <cooperative_groups.h>

#include "kv_cache.cuh"
#include "tree_launch.h"

namespace ssa {

struct TreeParams {
    int B, T, H, Hkv, S, depth, words, slices;
    const uint16_t *Q;
    const uint8_t *ck, *cv, *sk, *sv;
    const int32_t *len, *nodes, *parent;
    const uint64_t *dbits, *cbits, *goffs, *gcols;
    const int32_t *off_rank, *col_rank, *off_ptr, *offs, *col_ptr, *cols, *head_ptr, *heads;
    float scale_log2;
    uint16_t *O;
    float *LSE;
    int32_t *status;
    int64_t wait_ns;  // limit of a wait inside a kernel
};

namespace {

namespace cg = cooperative_groups;

// Entries below x of a merged list: the rank of x's word and the bits under x.
__device__ __forceinline__ int entries_below(const uint64_t *bits, const int32_t *rank, int x) {
    return __ldg(rank + (x >> 6)) + __popcll(__ldg(bits + (x >> 6)) & ((1ull << (x & 63)) - 1));
}

__device__ __forceinline__ uint64_t bit_window(const uint64_t *row, int o) {
    const uint64_t a = __ldg(row + (o >> 6)), b = __ldg(row + (o >> 6) + 1);
    const int s = o & 63;
    return s ? (a >> s) | (b << (64 - s)) : a;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// N consecutive words, N a power of two, aligned to min(N, 4) words.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *src, uint32_t (&w)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src) + i);
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
        }
    } else if constexpr (N == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
        w[0] = x.x;
        w[1] = x.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(src));
    }
}

// A run of elements of a stored row in a lane's registers: the words and the scale byte.
template <int FMT, int N>
struct Run {
    static constexpr int kWords = FMT == SSA_KV_BF16 ? N / 2 : FMT == SSA_KV_E4M3 ? N / 4 : N / 8;
    uint32_t w[kWords];
    uint32_t E;

    // row: within the (sequence, KV head) that the pointers start at
    __device__ __forceinline__ void load(const uint8_t *rows, const uint8_t *scales, uint32_t row, int d, int at) {
        load_words<kWords>(rows + static_cast<uint64_t>(row) * kv_row_bytes(FMT, d) + at * kWords * 4, w);
        if constexpr (FMT != SSA_KV_BF16)
            E = __ldg(scales + static_cast<uint64_t>(row) * (d / SSA_KV_GROUP) + at * N / SSA_KV_GROUP);
    }
    // bf16 pairs 2i and 2i + 1 (elements 4i .. 4i + 3)
    __device__ __forceinline__ void pairs(int i, uint32_t &a, uint32_t &b) const {
        if constexpr (FMT == SSA_KV_BF16) {
            a = w[2 * i];
            b = w[2 * i + 1];
        } else if constexpr (FMT == SSA_KV_E4M3) {
            decode_e4m3(w[i], kv_factor<FMT>(E), a, b);
        } else {
            decode_e2m1(w[i / 2] >> (16 * (i & 1)), kv_factor<FMT>(E), a, b);
        }
    }
    // element e as fp32
    __device__ __forceinline__ float value(int e) const {
        const int pair = FMT == SSA_KV_E4M3 ? e & 1 : (e >> 1) & 1, half = FMT == SSA_KV_E4M3 ? (e >> 1) & 1 : e & 1;
        uint32_t x[2];
        pairs(e / 4, x[0], x[1]);
        return half ? __uint_as_float(x[pair] & 0xffff0000u) : __uint_as_float(x[pair] << 16);
    }
};

// Weights that become fp16 are kept 2^kLift times as large: at most 2^(kSlack + kLift) = 2^15, and what
// falls below fp16's range is 2^-32 of the largest weight.
constexpr float kSlack = 8.0f;  // a reference moves when a logit (log2 domain) exceeds it by more
template <bool HALF>
constexpr float kLift = HALF ? 7.0f : 0.0f;

// Codes as fp16 pairs.  The hardware converts codes to fp16 (kv_cache.cuh's bf16 decoding takes
// twice the instructions), and 2^(E - 127) keeps every code exact in fp16 for E in
// [113, kv_scale_max].  Groups of zeros or with no value above 448 * 2^-15 (e4m3) or 6 * 2^-15
// (e2m1) lie below; they are decoded to bf16, exact for every scale, and multiplied as a bf16
// cache's: the step that has one, or the list of a CTA with tensor-memory tiles.
constexpr uint32_t kScaleHalf = 113;  // the smallest scale byte of the fp16 products
__device__ __forceinline__ uint32_t half_factors(uint32_t E0, uint32_t E1) {
    return ((E0 | (E1 << 16)) << 10) - 112u * 1024u * 0x10001u;
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// the two e4m3 codes in the low half of x
__device__ __forceinline__ uint32_t half_e4m3(uint32_t x) {
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(x));
    return d;
}

// the two e2m1 codes in each of the four bytes of x
__device__ __forceinline__ void half_e2m1(uint32_t x, uint32_t (&d)[4]) {
    asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, e;\n\t}"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(x));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The rows of one (sequence, KV head).
struct Rows {
    const uint8_t *k, *v, *ks, *vs;
};

template <int D, int FMT>
__device__ __forceinline__ Rows rows_of(const TreeParams &p, int b, int g) {
    const size_t row = (static_cast<size_t>(b) * p.Hkv + g) * p.S;
    Rows r;
    r.k = p.ck + row * kv_row_bytes(FMT, D);
    r.v = p.cv + row * kv_row_bytes(FMT, D);
    r.ks = p.sk + row * (D / SSA_KV_GROUP);
    r.vs = p.sv + row * (D / SSA_KV_GROUP);
    return r;
}

// The problem a CTA works on.
struct Problem {
    const int32_t *heads;         // of the group
    const int2 *offs, *cols;      // its lists
    const uint64_t *gcols;        // its columns as bits
    int n_off, n_col, len, nn, G;
    int first, last;              // rows of this CTA
    int head16[16];               // the first 16 heads
};

__device__ __forceinline__ int head_of(const Problem &w, int hh) { return hh < 16 ? w.head16[hh] : __ldg(w.heads + hh); }

// The tree of a sequence.
struct TreeInfo {
    uint64_t anc[SSA_TREE_MAX];  // node and its ancestors
    int jump[SSA_TREE_MAX];
    unsigned long long at_depth[SSA_TREE_MAX];  // the nodes of a depth
    uint8_t depth[SSA_TREE_MAX];
    int bad, max_depth;
};

// Ancestors and depths by pointer doubling: after k rounds a node knows its 2^k nearest.
__device__ __forceinline__ void resolve_tree(const TreeParams &p, TreeInfo &sh, int b, int nn) {
    const int n = threadIdx.x;
    if (n < SSA_TREE_MAX) sh.at_depth[n] = 0;
    if (n < nn) {
        int par = n - 1;
        if (p.parent) par = __ldg(p.parent + static_cast<size_t>(b) * p.T + n);
        if (par < -1 || par >= n) {
            sh.bad = 1;
            par = -1;
        }
        sh.anc[n] = 1ull << n;
        sh.jump[n] = par;
    }
    __syncthreads();
    for (int have = 1; have < nn; have <<= 1) {
        uint64_t a = 0;
        int j = -1;
        if (n < nn) {
            a = sh.anc[n];
            j = sh.jump[n];
            if (j >= 0) {
                a |= sh.anc[j];
                j = sh.jump[j];
            }
        }
        __syncthreads();
        if (n < nn) {
            sh.anc[n] = a;
            sh.jump[n] = j;
        }
        __syncthreads();
    }
    if (n < nn) {
        const int t = __popcll(sh.anc[n]) - 1;
        sh.depth[n] = static_cast<uint8_t>(t);
        atomicOr(&sh.at_depth[t], 1ull << n);
        if (t >= p.depth) sh.bad = 1;
        atomicMax(&sh.max_depth, t);
    }
}

// Which of the depths 0 .. 63 of a head retain a committed key at offset o.
__device__ __forceinline__ uint64_t look_up(const TreeParams &p, int h, int key, int o) {
    const uint64_t c = __ldg(p.cbits + static_cast<size_t>(h) * p.words + (key >> 6)) >> (key & 63);
    const uint64_t w = bit_window(p.dbits + static_cast<size_t>(h) * p.words, o);
    return (c & 1) ? ~0ull : w;
}

// An entry of the list on its way to a cache row and row bits, in three steps so that each
// step's load can be under way before the next: the list entry (fetch), the word of the
// group's columns that tells whether a band key is listed among them (probe), the rest.
struct Entry {
    int2 x;
    uint64_t c;
    int e;

    __device__ __forceinline__ void fetch(const Problem &w, int e_) {
        e = e_;
        x = make_int2(0, 0);
        if (e < w.n_off) x = __ldg(w.offs + e);
        else if (e < w.n_off + w.n_col) x = __ldg(w.cols + e - w.n_off);
    }
    __device__ __forceinline__ void probe(const Problem &w) {
        c = e < w.n_off ? __ldg(w.gcols + ((w.len - x.x) >> 6)) : 0;
    }

    // What the entry stands for: cache row j (or -1), its offset from len, the node whose row
    // it is (or -1), and the marks: bit k = head k retains it at all depths, 16 + k = it may.
    __device__ __forceinline__ void place(const Problem &w, int &j, int &o, int &node, uint32_t &marks) const {
        node = -1;
        marks = static_cast<uint32_t>(x.y);
        o = x.x;
        j = w.len - o;
        if (e < w.n_off) {
            if ((c >> (j & 63)) & 1) j = -1;  // listed among the columns
        } else if (e < w.n_off + w.n_col) {
            j = x.x;
            o = w.len - j;
            marks |= 0xffff0000u;  // a head without the column may still have the diagonal
        } else {
            node = e - w.n_off - w.n_col;
            j = node < w.nn ? w.len + node : -1;
        }
    }
};

// The nodes whose cache rows row r retains: of its ancestors and itself, those at a diagonal's
// distance or in a column of its head.
__device__ __forceinline__ uint64_t retained_nodes(const TreeParams &p, const Problem &w, const TreeInfo &tree, int r) {
    const int hh = r / w.nn, n = r - hh * w.nn;
    const size_t row = static_cast<size_t>(head_of(w, hh)) * p.words;
    const uint64_t diag = __ldg(p.dbits + row), col = bit_window(p.cbits + row, w.len);
    const int t = tree.depth[n];
    uint64_t kept = 0;
    for (uint64_t up = tree.anc[n]; up; up &= up - 1) {
        const int a = __ffsll(static_cast<long long>(up)) - 1, ta = tree.depth[a];
        kept |= (((diag >> (t - ta)) | (col >> ta)) & 1) << a;
    }
    return kept;
}

// The rows' node masks turned into the nodes' row masks: bit l of out[a] = lane l retains node a.
__device__ __forceinline__ void transpose_nodes(uint64_t kept, int nn, uint32_t *out) {
    const int lane = threadIdx.x & 31;
    uint32_t lo = 0, hi = 0;
    for (int a = 0; a < min(nn, 32); ++a) {
        const uint32_t rows = __ballot_sync(0xffffffffu, (kept >> a) & 1);
        if (lane == a) lo = rows;
    }
    for (int a = 32; a < nn; ++a) {
        const uint32_t rows = __ballot_sync(0xffffffffu, (kept >> a) & 1);
        if (lane == a - 32) hi = rows;
    }
    out[lane] = lo;
    out[32 + lane] = hi;
}

// Row bits of a CTA (WORDS x 32): bit i of word k = row first + 32 k + i.
template <int WORDS>
struct RowBits {
    uint32_t v[WORDS];

    // the rows of head hh at the nodes m
    __device__ __forceinline__ void add(const Problem &w, int hh, uint64_t m) {
        const int r0 = hh * w.nn - w.first;  // row of the head's node 0
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            const int s = r0 - 32 * k;
            if (s > -64 && s < 32) v[k] |= static_cast<uint32_t>(s >= 0 ? m << s : m >> -s);
        }
    }
    // the rows of head hh at the depths t
    __device__ __forceinline__ void add_depths(const Problem &w, const TreeInfo &tree, int hh, uint64_t t) {
        uint64_t m = 0;
        for (t &= (2ull << tree.max_depth) - 1; t; t &= t - 1) m |= tree.at_depth[__ffsll(static_cast<long long>(t)) - 1];
        add(w, hh, m);
    }
    // the rows that retain committed key j at offset o, of the heads in `some` (of the first 16)
    // and from the 17th on; four heads' loads at a time
    __device__ __forceinline__ void look_up_heads(const TreeParams &p, const Problem &w, const TreeInfo &tree,
                                                  uint32_t some, int j, int o) {
        while (some) {
            int hh[4];
            uint64_t t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                hh[k] = some ? __ffs(some) - 1 : -1;
                some &= some - 1;
                t[k] = hh[k] >= 0 ? look_up(p, w.head16[hh[k]], j, o) : 0;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t[k]) add_depths(w, tree, hh[k], t[k]);
        }
        if (w.G > 16) {  // heads without marks
            for (int hh = max(16, w.first / w.nn); hh * w.nn < w.last; ++hh)
                add_depths(w, tree, hh, look_up(p, __ldg(w.heads + hh), j, o));
        }
    }
};

// The look-ups of a committed key j at offset o, for the heads in `some`: up to four heads'
// words are loaded ahead, the rest (more than four, or heads without marks) when they are added.
struct LookUps {
    uint64_t c[4], a[4], b[4];
    uint32_t first, rest;

    __device__ __forceinline__ void load(const TreeParams &p, const Problem &w, uint32_t some, int j, int o) {
        first = some;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = a[k] = b[k] = 0;
            if (some) {
                const size_t row = static_cast<size_t>(w.head16[__ffs(some) - 1]) * p.words;
                c[k] = __ldg(p.cbits + row + (j >> 6));
                a[k] = __ldg(p.dbits + row + (o >> 6));
                b[k] = __ldg(p.dbits + row + (o >> 6) + 1);
                some &= some - 1;
            }
        }
        rest = some;
    }
    template <int WORDS>
    __device__ __forceinline__ void add(RowBits<WORDS> &v, const TreeParams &p, const Problem &w, const TreeInfo &tree, int j,
                                        int o) const {
        uint32_t some = first;
        const int s = o & 63;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!some) break;
            uint64_t t = s ? (a[k] >> s) | (b[k] << (64 - s)) : a[k];
            if ((c[k] >> (j & 63)) & 1) t = ~0ull;
            if (t) v.add_depths(w, tree, __ffs(some) - 1, t);
            some &= some - 1;
        }
        if (rest || w.G > 16) v.look_up_heads(p, w, tree, rest, j, o);
    }
};

// Slices of a launch of `items` problems, at most `most` each, by what the device runs at once.
template <class Kernel>
int pick_slices(Kernel kernel, cudaLaunchConfig_t cfg, ClusterCounts &counts, int device, long long items, int most) {
    return pick_slices(counts, device, items, most, [&](int k) {
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = k;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3(k);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
        cudaGetLastError();
        return -1;
    });
}

// The problem of a CTA, but for the list lengths, and those.
__device__ __forceinline__ void set_problem(const TreeParams &p, Problem &w, int g, int len, int nn, int first, int last,
                                            int hp, int G) {
    w.heads = p.heads + hp;
    w.offs = reinterpret_cast<const int2 *>(p.offs) + __ldg(p.off_ptr + g);
    w.cols = reinterpret_cast<const int2 *>(p.cols) + __ldg(p.col_ptr + g);
    w.gcols = p.gcols + static_cast<size_t>(g) * p.words;
    w.len = len, w.nn = nn, w.G = G;
    w.first = first, w.last = last;
}
__device__ __forceinline__ void set_heads(const TreeParams &p, Problem &w, int hp, int G, int k) {  // k = 0 .. 15
    w.head16[k] = k < G ? __ldg(p.heads + hp + k) : 0;
}
__device__ __forceinline__ void set_lengths(const TreeParams &p, Problem &w, int g, int len, bool bad) {
    if (bad) {  // no list entry is looked at
        w.n_off = w.n_col = 0;
        return;
    }
    const size_t at = static_cast<size_t>(g) * p.words;
    w.n_off = entries_below(p.goffs + at, p.off_rank + at, len + 1);
    w.n_col = entries_below(p.gcols + at, p.col_rank + at, len);
}

// Index of row r = (head of the group, node) in Q, O and LSE.
__device__ __forceinline__ size_t row_index(const TreeParams &p, const Problem &w, int b, int r) {
    const int hh = r / w.nn;
    return (static_cast<size_t>(b) * p.T + (r - hh * w.nn)) * p.H + head_of(w, hh);
}

// Joins the parts of the rows [first, last), one warp a row; lane k holds the factor of part
// k = (slice, one of PER_CTA).  ml(c, i): reference (log2 domain) and sum of row i in part c of
// this CTA, part(c, i): its O, in shared memory that every CTA of the cluster lays out alike.
template <int D, int PER_CTA, class ML, class PART>
__device__ __forceinline__ void join_parts(const TreeParams &p, const Problem &w, int b, int slice, int warp, int warps,
                                           ML ml, PART part) {
    constexpr int EPL = D / 32;
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, n_parts = p.slices * PER_CTA;
    for (int r = w.first + slice * warps + warp; r < w.last; r += p.slices * warps) {
        const int i = r - w.first;
        float m = -INFINITY, l = 0.0f;
        if (lane < n_parts) {
            const float *src = ml(lane % PER_CTA, i);
            if (p.slices > 1) src = cluster.map_shared_rank(src, lane / PER_CTA);
            m = src[0];
            l = src[1];
        }
        float top = m;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float f = m == top ? 1.0f : ex2_approx(m - top);  // a lane without a part: 0
        float sum = lane < n_parts ? f * l : 0.0f;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        float a[EPL] = {};
        // eight parts at a time, all their loads before the sums: a distributed load takes
        // most of a microsecond
        for (int k0 = 0; k0 < n_parts; k0 += 8) {
            float v[8][EPL];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int k = k0 + u;
#pragma unroll
                for (int e = 0; e < EPL; ++e) v[u][e] = 0.0f;
                if (k < n_parts) {
                    const float *src = part(k % PER_CTA, i) + EPL * lane;
                    if (p.slices > 1) src = cluster.map_shared_rank(src, k / PER_CTA);
                    if constexpr (EPL == 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(src);
                        v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2 *>(src);
                        v[u][0] = x.x, v[u][1] = x.y;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float fk = __shfl_sync(0xffffffffu, f, (k0 + u) & 31);
                if (k0 + u < n_parts) {
#pragma unroll
                    for (int e = 0; e < EPL; ++e) a[e] = fmaf(fk, v[u][e], a[e]);
                }
            }
        }
        const bool empty = sum == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / sum;
        const size_t out = row_index(p, w, b, r);
#pragma unroll
        for (int k = 0; k < EPL; k += 2)
            *reinterpret_cast<uint32_t *>(p.O + out * D + EPL * lane + k) = pack_bf16(a[k] * inv, a[k + 1] * inv);
        if (lane == 0) p.LSE[out] = empty ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    }
}

// Power of two that brings a query row's largest finite element (bf16 bits without sign) to
// [2^14, 2^15), at most 2^60: what then falls below fp16's range is under 2^-38 of it.
__device__ __forceinline__ int query_shift(uint32_t top) { return min(14 - (static_cast<int>(top >> 7) - 127), 60); }

__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float(static_cast<uint32_t>(127 + n) << 23); }

// Logit (log2 domain) per unit of the products of a query row shifted by `up`: not zero, with which
// the -inf of a key that the row does not retain would be NaN (such products are under 2^38, so
// that the logits are zero to fp32 either way).
__device__ __forceinline__ float shifted_scale(float scale_log2, int up) {
    return fmaxf(scale_log2 * power_of_two(-up), 1.17549435e-38f);
}

}  // namespace

// KV heads of more rows than attn_tree_kernel takes (tree_wide.cu).
int launch_tree_wide(TreeParams &p, int d, int fmt, int rows, int entries, cudaStream_t s);

}  // namespace ssa
