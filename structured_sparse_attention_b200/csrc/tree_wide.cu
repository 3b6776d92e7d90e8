// tree_wide.cu -- the tree attention where a KV head has many rows (query heads of the group
// x nodes): products on tcgen05 with accumulators in tensor memory.
//
// A CTA takes 128 rows and its share of the key list in tiles of 64 keys:
//   warps 12, 13  resolve the tiles' list entries ahead (cache rows, row bits)
//   warp 15       turns the entries' row bits to key bits of each row
//   warps 4-11    gather a tile's key and value rows into registers (the next tile's loads are
//                 issued before this one is worked on) and decode them to 16-bit tiles in
//                 shared memory (128-byte swizzle: K rows K-major; the same layout read with
//                 the keys as inner index for V); four lanes a row (eight, with loads of whole
//                 runs and stores free of bank conflicts, measured 5 % slower)
//   warp 14       one lane issues S = Q K^T (128 x 64) of tile i, then O += P V of tile i - 1
//   warps 0-3     softmax, one thread a row: S from tensor memory, key bits, running maximum and
//                 sum in fp32 (log2 domain), P back into S's columns as the next A operand; O is
//                 rescaled only when a reference grows by over 2^8
// Resolved entries have a ring of eight tiles, so that the gathers run ahead; the staged rows, S
// and P a ring of four.  Barriers: resolved, turned, entry_free; full (rows staged), s_full (S there),
// p_full (P there), pv_done (P V done: the slot is free).  Every wait follows the same waiter's
// observation of the barrier's phase before, and no barrier can run two phases ahead of a
// waiter, so a parity stands for one phase only.
//
// Quantised caches become fp16 tiles (every code is exact while the scale is in fp16's
// range) and P is fp16; bf16 caches stay bf16 and P is split into two bf16 (see tree.cu).  A
// CTA that meets a group below that range (but for zeros) gives its pass up and takes its list
// again with bf16 tiles, in code out of line: 16 trees of 64 nodes over 1000 e4m3 keys 62 us, 103 with
// values of deviation 0.005, at most about 130 where the only small group is the last (key by key such
// values took 14.7 ms).  Both kinds of tile in one loop cost the usual ones 15 %, bf16 tiles for
// all 11 % (37 % on lists of 7400 keys).  A key with a value that is not finite is taken out of
// the tile (zeros, no row bits) and added in fp32 by the rows that retain it.
//
// One CTA of 16 warps an SM, each role in warps of its own: with resolving, decoding and
// issuing in one group of four warps and two CTAs an SM, every step of the chain waited for
// the one before and a tile took 2.3 us of an SM.  Two threads a row (32 keys each, 20 warps), or
// two groups of softmax warps on alternate tiles with an O each, measured slower (16 trees of
// 64 nodes over 7400 keys: 401 and 460 us against 358): the roles' code contends for the
// instruction caches, not for the units.
//
// Measured, d = 128: 16 trees of 64 nodes, 32 query heads on 8, e4m3, lists of about 1000 keys:
// 62 us.  The tiles' products alone, masked pairs included, would take 7 us at the card's bf16 rate
// (tensor pipe 8 % busy); a tile takes 2500 to 3000 cycles, most of them the softmax of 64 keys a
// row by one warp a scheduler (a sixth of the working warps' stalls wait for instructions to be
// fetched), and 256 CTAs on 148 SMs make two waves.  4 trees of 16 nodes over 104000 rows, bf16:
// 55 us.
#include <atomic>

#include "trace.h"
#include "tree.cuh"

namespace ssa {
namespace {

constexpr int kM = 128, kN = 64;         // rows, keys of a tile
constexpr int kProducers = 256, kResolvers = 64, kRing = 4, kEntries = 8;
constexpr int kThreads = 512;
constexpr int kWarpProduce = 4, kWarpResolve = 12, kWarpMma = 14, kWarpTurn = 15;
constexpr uint32_t kTmemCols = 512;      // S, P: kRing x 64, O: d
constexpr uint32_t kColO = kRing * kN;
constexpr int64_t kDrainNs = 1000000000LL;

template <int D>
struct Wide {
    static constexpr int kPanels = D / 64;                  // of 64 elements: 128-byte rows
    static constexpr int kQ = kPanels * kM * 128;           // bytes
    static constexpr int kTile = kPanels * kN * 128;
    static constexpr int kPartPitch = D + 4;                // floats
    static constexpr int kUsed = kQ + 2 * kRing * kTile;    // Q, kRing x (K, V); later the rows' part
    static constexpr int kPart = kM * kPartPitch * 4;
    // At least 120 KB, so that two CTAs never share an SM: the second would wait for tensor
    // memory while its cluster waits for it.
    static constexpr int kMin = 120 * 1024;
    static constexpr int kBig = kUsed > kPart ? kUsed : kPart;
    static constexpr int kBytes = (kBig > kMin ? kBig : kMin) + 1024;  // + alignment
};

struct Barriers {
    uint64_t resolved[kEntries], turned[kEntries], entry_free[kEntries];
    uint64_t full[kRing], s_full[kRing], p_full[kRing], pv_done[kRing], drain;
};

struct WideShared : TreeInfo {
    Barriers bars[2];  // of the first and of a second pass
    uint32_t tmem;
    int abort;
    int small;  // the pass met a group below fp16's exact range
    // ring of resolved tiles; mask: bit i of word w = row first + 32 w + i retains the key
    int key[kEntries][kN];
    uint32_t mask[kEntries][4][kN];
    uint32_t keys[kEntries][2][kM];  // the same turned: bit k of a row's word h = it retains key 32 h + k
    uint8_t odd[kRing][kN];          // keys taken out of a tile
    uint32_t here;                   // heads (of the first 16) with rows in [first, last)
    uint4 spread[4][16];             // rows of four heads' bits
    uint32_t node_rows[4][64];       // rows that retain a node
    float ml[kM][2];
    Problem w;
};

// Shared-memory matrix descriptor, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor, kind::f16: A and B both bf16 or both fp16, fp32 accumulation, A K-major.
__host__ __device__ constexpr uint32_t instr_desc(bool bf, int N, bool b_mn_major) {
    return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | ((b_mn_major ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kM >> 4) << 24);
}

// A bounded wait of warps that run ahead of the others: asleep between polls, so that they
// leave the issue slots to the softmax warps on the same scheduler.
__device__ __forceinline__ bool wait_asleep(uint64_t *bar, int parity, int64_t limit_ns, volatile int *abort) {
    if (mbar_test(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        __nanosleep(200);
        if (mbar_test(bar, parity)) return true;
        if (*abort || static_cast<int64_t>(global_timer_ns() - t0) >= limit_ns) return false;
    }
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A 32 x 32 bit matrix, a row a lane, transposed: five exchanges of halves, quarters, ..
__device__ __forceinline__ uint32_t transpose32(uint32_t x) {
    const int lane = threadIdx.x & 31;
    uint32_t low = 0x0000ffffu;  // the columns whose bit `d` is clear
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const uint32_t y = __shfl_xor_sync(0xffffffffu, x, d);
        x = (lane & d) ? (x & ~low) | ((y >> d) & low) : (x & low) | ((y << d) & ~low);
        low ^= low << (d >> 1);
    }
    return x;
}

// 32 lanes x 8 columns of tensor memory.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// A quarter of a stored row (D/4 elements) in registers, decoded to 16-bit chunks of 8 elements.
template <int D, int FMT>
struct Quarter {
    static constexpr int kWords = FMT == SSA_KV_BF16 ? D / 8 : FMT == SSA_KV_E4M3 ? D / 16 : D / 32;
    uint32_t w[kWords];
    uint32_t E;  // one scale group at most

    __device__ __forceinline__ void load(const uint8_t *rows, const uint8_t *scales, uint32_t row, int quarter) {
        load_words<kWords>(rows + static_cast<uint64_t>(row) * kv_row_bytes(FMT, D) + quarter * kWords * 4, w);
        if constexpr (FMT != SSA_KV_BF16)
            E = __ldg(scales + static_cast<uint64_t>(row) * (D / SSA_KV_GROUP) + quarter * (D / 4) / SSA_KV_GROUP);
    }
    // not finite: the key is taken out of its tile
    __device__ __forceinline__ bool odd(bool value) const {
        if constexpr (FMT == SSA_KV_BF16) {
            if (!value) return false;  // a key's infinities and NaN stay in its own logits
            uint32_t c = 0;            // x * 0 is NaN for an infinity or a NaN, and stays one
#pragma unroll
            for (int i = 0; i < kWords; ++i) c = bf2_fma(w[i], 0u, c);
            return (c & 0x7fff7fffu) != 0;
        } else {
            return E > kv_scale_max(FMT);
        }
    }
    // below fp16's exact range, and not all zero
    __device__ __forceinline__ bool small() const {
        if (FMT == SSA_KV_BF16 || E >= kScaleHalf) return false;
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i) c |= w[i];
        return (c & (FMT == SSA_KV_E4M3 ? 0x7f7f7f7fu : 0x77777777u)) != 0;
    }

    template <bool HALF>
    __device__ __forceinline__ uint4 chunk(int j) const {
        uint32_t d[4];
        if constexpr (FMT == SSA_KV_BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = w[4 * j + i];
        } else if constexpr (!HALF) {
            const uint32_t f = kv_factor<FMT>(E);
            if constexpr (FMT == SSA_KV_E4M3) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t even, odd;
                    decode_e4m3(w[2 * j + i], f, even, odd);
                    d[2 * i] = prmt(even, odd, 0x5410u);
                    d[2 * i + 1] = prmt(even, odd, 0x7632u);
                }
            } else {
                decode_e2m1(w[j], f, d[0], d[1]);
                decode_e2m1(w[j] >> 16, f, d[2], d[3]);
            }
        } else {
            const uint32_t e = max(E, kScaleHalf), f = half_factors(e, e);  // a lower E has codes of zero
            if constexpr (FMT == SSA_KV_E4M3) {
                d[0] = half_e4m3(w[2 * j]);
                d[1] = half_e4m3(w[2 * j] >> 16);
                d[2] = half_e4m3(w[2 * j + 1]);
                d[3] = half_e4m3(w[2 * j + 1] >> 16);
            } else {
                half_e2m1(w[j], d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = h2_mul(d[i], f);
        }
        return make_uint4(d[0], d[1], d[2], d[3]);
    }
    // to the row of a tile; zeros where the key is taken out
    template <bool HALF>
    __device__ __forceinline__ void stage(uint8_t *tile, int key, int quarter, bool keep) const {
        constexpr int kChunks = D / 32;  // of this quarter
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            const int c = (quarter * kChunks + j) & 7, panel = (quarter * kChunks + j) >> 3;
            const uint4 v = keep ? chunk<HALF>(j) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(tile + panel * (kN * 128) + key * 128 + ((c ^ (key & 7)) << 4)) = v;
        }
    }
};

// The work of a CTA, with fp16 tiles (HALF) or bf16 ones.  False, with no output and the tensor memory
// still held, if a pass with fp16 tiles met a group below their exact range.
template <int D, int FMT, bool HALF>
__device__ __forceinline__ bool attend(const TreeParams &p, WideShared &sh, uint8_t *smem) {
    using C = Wide<D>;
    constexpr bool kFirst = HALF || FMT == SSA_KV_BF16;  // else after such a pass
    Barriers &bars = sh.bars[kFirst ? 0 : 1];
    uint8_t *const s_q = smem, *const s_kv = smem + C::kQ;  // stage s: K at 2 s kTile, V behind it
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slice = blockIdx.x % p.slices, first = (blockIdx.x / p.slices) * kM;
    const int g = blockIdx.y, b = blockIdx.z;
    cg::cluster_group cluster = cg::this_cluster();

    const int len = __ldg(p.len + b);
    int nn = p.nodes ? __ldg(p.nodes + b) : p.T;
    const int hp = __ldg(p.head_ptr + g), G = __ldg(p.head_ptr + g + 1) - hp;
    bool bad = len < 0 || nn < 0 || nn > p.T || static_cast<long long>(len) + nn > p.S;
    nn = min(max(nn, 0), p.T);
    if (first >= G * nn) {  // every CTA of the cluster alike
        if (bad && g == 0 && first == 0 && slice == 0 && tid == 0) report(p.status, SSA_ERR_INVALID);
        return true;
    }
    const int last = min(first + kM, G * nn);
    if (tid == 0) {
        sh.bad = bad;
        sh.max_depth = 0;
        sh.abort = sh.small = 0;
        set_problem(p, sh.w, g, len, nn, first, last, hp, G);
        uint32_t here = 0;
        for (int hh = first / nn; hh < 16 && hh * nn < last; ++hh) here |= 1u << hh;
        sh.here = here;
        for (int s = 0; s < kEntries; ++s) {
            mbar_init(&bars.resolved[s], kResolvers);
            mbar_init(&bars.turned[s], 32);
            mbar_init(&bars.entry_free[s], 1);
        }
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&bars.full[s], kProducers);
            mbar_init(&bars.s_full[s], 1);
            mbar_init(&bars.p_full[s], kM);
            mbar_init(&bars.pv_done[s], 1);
        }
        mbar_init(&bars.drain, 1);
        fence_barrier_init();
    } else if (tid == 32) {
        set_lengths(p, sh.w, g, len, bad);
    } else if (tid >= 64 && tid < 128) {
        const int set = (tid - 64) >> 4;
        uint32_t rows[4] = {0, 0, 0, 0};
        for (int k = 0; k < 4; ++k) {
            const int lo = max((4 * set + k) * nn, first), hi = min((4 * set + k + 1) * nn, last);
            if (!((tid >> k) & 1)) continue;
            for (int w = 0; w < 4; ++w) {  // rows [lo, hi) of word w
                const int a = max(lo - first - 32 * w, 0), z = min(hi - first - 32 * w, 32);
                if (a < z) rows[w] |= (0xffffffffu >> (32 - (z - a))) << a;
            }
        }
        sh.spread[set][tid & 15] = make_uint4(rows[0], rows[1], rows[2], rows[3]);
    }
    if (tid >= 128 && tid < 144) set_heads(p, sh.w, hp, G, tid - 128);
    if (kFirst && warp == kWarpMma) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    __syncthreads();
    const Problem &w = sh.w;
    // what needs no more than the lengths of the lists is loaded while the tree is worked out:
    // the rows of Q, the first list entries
    const int row = first + (tid & (kM - 1));  // warps 0-3 (and 4-7 for the nodes' rows)
    const uint16_t *q_row = nullptr;
    uint4 v[D / 8];
    Entry now, next, after;
    const int e_own = slice * kN + tid - 32 * kWarpResolve;  // of the resolvers
    if (tid < kM) {
        if (row < last) q_row = p.Q + row_index(p, w, b, row) * D;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            v[c] = make_uint4(0, 0, 0, 0);
            if (q_row) v[c] = __ldg(reinterpret_cast<const uint4 *>(q_row) + c);
        }
    } else if (warp >= kWarpResolve && warp < kWarpMma) {
        now.fetch(w, e_own);
        next.fetch(w, e_own + p.slices * kN);
        after.fetch(w, e_own + 2 * p.slices * kN);
        now.probe(w);
        next.probe(w);
    }
    resolve_tree(p, sh, b, nn);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    // Q's rows into shared memory, O to zero
    float scale = p.scale_log2, shift = 1.0f;
    if (tid < kM) {
        if (HALF) {
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint32_t u[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = u[i] & 0x7fffu, hi = (u[i] >> 16) & 0x7fffu;
                    top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                }
            }
            const int up = query_shift(top);
            shift = power_of_two(up);
            scale = shifted_scale(scale, up);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            if (HALF) {
                uint32_t u[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    u[i] = pack_half(__uint_as_float(u[i] << 16) * shift, __uint_as_float(u[i] & 0xffff0000u) * shift);
                v[c] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            *reinterpret_cast<uint4 *>(s_q + (c >> 3) * (kM * 128) + tid * 128 + (((c & 7) ^ (tid & 7)) << 4)) = v[c];
        }
        fence_async_shared();
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_st32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + kColO + 32 * c, z);
        tmem_wait_st();
        tc_fence_before();
    } else if (tid < 2 * kM) {
        transpose_nodes(row < last && !bad ? retained_nodes(p, w, sh, row) : 0, nn, sh.node_rows[warp - 4]);
    }
    __syncthreads();
    bad = sh.bad;
    if (bad && slice == 0 && tid == 0) report(p.status, SSA_ERR_INVALID);
    tc_fence_after();

    const Rows rows = rows_of<D, FMT>(p, b, g);
    const int total = bad ? 0 : w.n_off + w.n_col + nn;
    const int tiles_all = (total + kN - 1) / kN;
    const int tiles = tiles_all > slice ? (tiles_all - slice + p.slices - 1) / p.slices : 0;  // slice, slice + slices, ..
    volatile int *abort = &sh.abort, *small = &sh.small;
    const auto give_up = [&] {  // after a wait that ended without its phase
        if (!HALF || !*small) report(p.status, SSA_ERR_TIMEOUT);
        *abort = 1;
    };
    const int64_t lim = p.wait_ns;
    float m = -3.402823466e38f, l = 0.0f;  // this row's reference (log2 domain) and sum

    if (warp == kWarpTurn) {
        // ------------------------------ row bits turned to key bits ------------------------------
        bool ok = true;
        for (int i = 0; i < tiles; ++i) {
            const int slot = i % kEntries;
            if (!__all_sync(0xffffffffu, wait_asleep(&bars.resolved[slot], (i / kEntries) & 1, lim, abort))) {
                ok = false;
                break;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (first + 32 * q >= last) break;
                sh.keys[slot][0][32 * q + lane] = transpose32(sh.mask[slot][q][lane]);
                sh.keys[slot][1][32 * q + lane] = transpose32(sh.mask[slot][q][32 + lane]);
            }
            mbar_arrive(&bars.turned[slot]);
        }
        if (!ok) give_up();
    } else if (warp >= kWarpResolve && warp < kWarpMma) {
        // ------------------------------ resolvers ------------------------------
        const int e = tid - 32 * kWarpResolve;
        // an entry is fetched three tiles ahead, probed two, its look-ups are loaded one ahead
        LookUps ahead;
        int j, o, node;
        uint32_t marks;
        const auto peek = [&](const Entry &x) {
            x.place(w, j, o, node, marks);
            ahead.load(p, w, j >= 0 && node < 0 ? (marks >> 16) & ~marks & sh.here : 0, j, o);
        };
        peek(now);
        bool ok = true;
        for (int i = 0; i < tiles; ++i) {
            const int j_now = j;
            RowBits<4> v{};
            if (j < 0) {
            } else if (node >= 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v.v[k] = sh.node_rows[k][node];
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (4 * k < w.G) {
                        const uint4 s = sh.spread[k][(marks >> (4 * k)) & 15];
                        v.v[0] |= s.x, v.v[1] |= s.y, v.v[2] |= s.z, v.v[3] |= s.w;
                    }
                }
                ahead.add(v, p, w, sh, j, o);
            }
            now = next;
            next = after;
            next.probe(w);
            after.fetch(w, e_own + (i + 3) * p.slices * kN);  // beyond the list: no key
            peek(now);
            const int slot = i % kEntries;
            if (i >= kEntries &&
                !__all_sync(0xffffffffu, wait_asleep(&bars.entry_free[slot], ((i - kEntries) / kEntries) & 1, lim, abort))) {
                ok = false;
                break;
            }
            // an entry that no row retains: the first node's row, which is there to be read
            sh.key[slot][e] = (v.v[0] | v.v[1] | v.v[2] | v.v[3]) ? j_now : w.len;
#pragma unroll
            for (int k = 0; k < 4; ++k) sh.mask[slot][k][e] = v.v[k];
            mbar_arrive(&bars.resolved[slot]);
        }
        if (!ok) give_up();
    } else if (warp >= kWarpProduce && warp < kWarpResolve) {
        // ------------------------------ producers ------------------------------
        const int pt = tid - 32 * kWarpProduce, key = pt >> 2, quarter = pt & 3;
        Quarter<D, FMT> kr, vr, kn, vn;
        bool ok = true;
        const auto load = [&](int i) {  // rows of tile i, once it is resolved
            ok = __all_sync(0xffffffffu, wait_asleep(&bars.resolved[i % kEntries], (i / kEntries) & 1, lim, abort));
            if (!ok) return;
            const int j = sh.key[i % kEntries][key];
            kn.load(rows.k, rows.ks, j, quarter);
            vn.load(rows.v, rows.vs, j, quarter);
        };
        if (tiles > 0) load(0);
        for (int i = 0; i < tiles && ok; ++i) {
            const int st = i % kRing;
            kr = kn;
            vr = vn;
            if (i + 1 < tiles) load(i + 1);
            if (!ok) break;
            if (i >= kRing && !__all_sync(0xffffffffu, wait_asleep(&bars.pv_done[st], ((i - kRing) / kRing) & 1, lim, abort))) {
                ok = false;
                break;
            }
            if constexpr (HALF) {
                if (__any_sync(0xffffffffu, kr.small() || vr.small())) {  // the pass ends
                    *small = 1;
                    ok = false;
                    break;
                }
            }
            bool odd = kr.odd(false) || vr.odd(true);
            odd = __shfl_xor_sync(0xffffffffu, odd, 1) || odd;
            odd = __shfl_xor_sync(0xffffffffu, odd, 2) || odd;
            if constexpr (FMT != SSA_KV_BF16)
                if (odd && (kv_bad_scale(FMT, kr.E) || kv_bad_scale(FMT, vr.E))) report(p.status, SSA_ERR_INVALID);
            uint8_t *tile = s_kv + 2 * st * C::kTile;
            kr.template stage<HALF>(tile, key, quarter, !odd);
            vr.template stage<HALF>(tile + C::kTile, key, quarter, !odd);
            if (quarter == 0) sh.odd[st][key] = odd;
            fence_async_shared();
            mbar_arrive(&bars.full[st]);
        }
        if (!ok) give_up();
    } else if (warp == kWarpMma) {
        // ------------------------------ MMA issuer ------------------------------
        if (lane == 0) {
            constexpr uint32_t kQK = instr_desc(!HALF, kN, false), kPV = instr_desc(!HALF, D, true);
            const uint32_t aq = smem_u32(s_q), akv = smem_u32(s_kv);
            bool ok = true;
            for (int i = 0; i <= tiles; ++i) {
                if (i < tiles) {
                    const int st = i % kRing;
                    if (!mbar_wait_poll(&bars.full[st], (i / kRing) & 1, lim, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ak = akv + 2 * st * C::kTile;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_ss(tmem + kN * st, smem_desc(aq + (k >> 2) * (kM * 128) + (k & 3) * 32, 16, 1024),
                                smem_desc(ak + (k >> 2) * (kN * 128) + (k & 3) * 32, 16, 1024), kQK, k > 0 ? 1u : 0u);
                    umma_commit(&bars.s_full[st]);
                }
                if (i > 0) {
                    const int st = (i - 1) % kRing;
                    if (!mbar_wait_poll(&bars.p_full[st], ((i - 1) / kRing) & 1, lim, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t av = akv + (2 * st + 1) * C::kTile;
#pragma unroll
                    for (int k = 0; k < kN / 16; ++k) {  // 16 keys: 16 rows of 128 bytes
                        const uint64_t dv = smem_desc(av + k * 2048, kN * 128, 1024);
                        umma_ts(tmem + kColO, tmem + kN * st + 8 * k, dv, kPV, 1u);
                        if (!HALF) umma_ts(tmem + kColO, tmem + kN * st + 32 + 8 * k, dv, kPV, 1u);
                    }
                    umma_commit(&bars.pv_done[st]);
                    umma_commit(&bars.entry_free[(i - 1) % kEntries]);
                }
            }
            if (!ok) give_up();
            umma_commit(&bars.drain);  // completes once every MMA issued is done
            mbar_wait(&bars.drain, 0, kDrainNs, nullptr);
        }
        __syncwarp();
    } else {
        // ------------------------------ softmax ------------------------------
        const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
        const uint32_t t_o = tmem + lanes + kColO;
        const bool any_row = first + 32 * warp < last;  // of this warp
        bool ok = true;
        const auto wait = [&](uint64_t *bar, int parity) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar, parity, lim, abort))) ok = false;
            return ok;
        };
        for (int i = 0; i < tiles; ++i) {
            const int st = i % kRing, before = (i + kRing - 1) % kRing;  // slots of tiles i, i - 1
            const int parity = (i / kRing) & 1, slot = i % kEntries;
            // (P V of tile i - kRing is done by then; observed here so that no wait on pv_done is ever
            // more than one phase behind)
            const bool there = mbar_test(&bars.full[st], parity) & mbar_test(&bars.s_full[st], parity) &
                               mbar_test(&bars.turned[slot], (i / kEntries) & 1) &
                               (i < kRing || mbar_test(&bars.pv_done[st], parity ^ 1));
            if (!__all_sync(0xffffffffu, there) &&
                (!wait(&bars.full[st], parity) || !wait(&bars.s_full[st], parity) ||
                 !wait(&bars.turned[slot], (i / kEntries) & 1) || (i >= kRing && !wait(&bars.pv_done[st], parity ^ 1))))
                break;
            tc_fence_after();
            if (any_row) {
                // keys taken out of the tile, in fp32: one by one, before the others
                const uint32_t special[2] = {__ballot_sync(0xffffffffu, sh.odd[st][lane]),
                                             __ballot_sync(0xffffffffu, sh.odd[st][lane + 32])};
                const bool some_special = (special[0] | special[1]) != 0;
                if (some_special) {
                    if (i > 0) {
                        if (!wait(&bars.pv_done[before], ((i - 1) / kRing) & 1)) break;
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int k = 0; k < 64; ++k) {
                        if (!((special[k >> 5] >> (k & 31)) & 1)) continue;
                        const bool in = q_row && ((sh.keys[slot][k >> 5][tid] >> (k & 31)) & 1);
                        const uint32_t j = sh.key[slot][k];
                        float dot = 0.0f;
#pragma unroll 1
                        for (int c = 0; in && c < D / 8; ++c) {
                            Run<FMT, 8> x;
                            x.load(rows.k, rows.ks, j, D, c);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dot = fmaf(__uint_as_float(static_cast<uint32_t>(__ldg(q_row + 8 * c + e)) << 16), x.value(e), dot);
                        }
                        __syncwarp();  // the loop ran in some lanes; tensor memory is read by the whole warp
                        const float y = in ? dot * p.scale_log2 : -INFINITY;
                        const float up = fmaxf(m, y - kLift<HALF>), f = up == m ? 1.0f : ex2_approx(m - up);
                        const float wt = in ? ex2_approx(y - up) : 0.0f;
                        m = up;
                        l = l * f + wt;
#pragma unroll 1
                        for (int c = 0; c < D; c += 8) {
                            Run<FMT, 8> x;
                            x.load(rows.v, rows.vs, j, D, c / 8);
                            uint32_t o[8];
                            tmem_ld8(t_o + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float old = __uint_as_float(o[e]) * f;
                                o[e] = __float_as_uint(in ? fmaf(wt, x.value(e), old) : old);
                            }
                            tmem_st8(t_o + c, o);
                        }
                        tmem_wait_st();
                    }
                }
                const uint32_t t_s = tmem + lanes + kN * st;
                uint32_t r[64];
                tmem_ld32(t_s, r);
                tmem_ld32(t_s + 32, r + 32);
                // a key that the row does not retain gets the logit -inf: no weight
                const uint32_t keys[2] = {sh.keys[slot][0][tid] & ~special[0], sh.keys[slot][1][tid] & ~special[1]};
                tmem_wait_ld();
                if (!__all_sync(0xffffffffu, (keys[0] & keys[1]) == 0xffffffffu || row >= last)) {
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (!((keys[k >> 5] >> (k & 31)) & 1)) r[k] = 0xff800000u;
                }
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < 64; k += 2) top = fmax3(top, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                top *= scale;
                if (__any_sync(0xffffffffu, top > m + (kSlack + kLift<HALF>))) {
                    const float up = fmaxf(top - kLift<HALF>, m), f = up == m ? 1.0f : ex2_approx(m - up);
                    m = up;
                    l *= f;
                    if (i > 0 || some_special) {  // else O is still zero
                        if (i > 0 && !some_special) {
                            if (!wait(&bars.pv_done[before], ((i - 1) / kRing) & 1)) break;
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[8], z[8];
                            tmem_ld8(t_o + c, o);
                            tmem_ld8(t_o + c + 8, z);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                z[e] = __float_as_uint(__uint_as_float(z[e]) * f);
                            }
                            tmem_st8(t_o + c, o);
                            tmem_st8(t_o + c + 8, z);
                        }
                        tmem_wait_st();
                    }
                }
                const uint64_t s2 = f2_pack(scale, scale), m2 = f2_pack(-m, -m);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int k = 0; k < 64; k += 4) {
                    float x[4];
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), s2, m2), x[0], x[1]);
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])), s2, m2), x[2], x[3]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[u] = ex2_approx(x[u]);
                    sum0 = f2_add(sum0, f2_pack(x[0], x[1]));
                    sum1 = f2_add(sum1, f2_pack(x[2], x[3]));
#pragma unroll
                    for (int u = 0; u < 4; ++u) r[k + u] = __float_as_uint(x[u]);
                }
                float a0, a1;
                f2_unpack(f2_add(sum0, sum1), a0, a1);
                l += a0 + a1;
                uint32_t hi[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float x = __uint_as_float(r[2 * k]), y = __uint_as_float(r[2 * k + 1]);
                    hi[k] = HALF ? pack_half(x, y) : pack_bf16(x, y);
                }
                tmem_st32(t_s, hi);
                if constexpr (!HALF) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        hi[k] = pack_bf16(__uint_as_float(r[2 * k]) - __uint_as_float(hi[k] << 16),
                                          __uint_as_float(r[2 * k + 1]) - __uint_as_float(hi[k] & 0xffff0000u));
                    tmem_st32(t_s + 32, hi);
                }
                tmem_wait_st();
                tc_fence_before();
            }
            mbar_arrive(&bars.p_full[st]);
        }
        // the last tile's P V
        if (ok && tiles > 0 && wait(&bars.pv_done[(tiles - 1) % kRing], ((tiles - 1) / kRing) & 1)) tc_fence_after();
        if (!ok) give_up();
    }
    // Every MMA is done (the issuer has waited for its own), Q and the tiles are no longer read.
    tc_fence_before();
    __syncthreads();
    if (HALF && *small) return false;
    tc_fence_after();
    float *part = reinterpret_cast<float *>(smem);
    if (warp < 4 && first + 32 * warp < last) {
        const uint32_t t_o = tmem + (static_cast<uint32_t>(32 * warp) << 16) + kColO;
        const bool direct = p.slices == 1, empty = l == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / l;
        const size_t out = row < last ? row_index(p, w, b, row) : 0;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t r[32];
            __syncwarp();  // after the stores of some lanes: the whole warp reads its columns
            tmem_ld32(t_o + c, r);
            tmem_wait_ld();
            if (direct) {  // the only part: the result
                if (row < last) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.O + out * D + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = pack_bf16(__uint_as_float(r[8 * k + 2 * e]) * inv, __uint_as_float(r[8 * k + 2 * e + 1]) * inv);
                        dst[k] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            } else {
                float4 *dst = reinterpret_cast<float4 *>(part + tid * C::kPartPitch + c);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dst[k] = make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                                         __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
            }
        }
        if (direct) {
            if (row < last) p.LSE[out] = empty ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
            sh.ml[tid][0] = m;
            sh.ml[tid][1] = l;
        }
        tc_fence_before();
    }
    if (p.slices > 1) cluster.sync();
    else __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (p.slices == 1) return true;
    join_parts<D, 1>(
        p, w, b, slice, warp, kThreads / 32, [&](int, int i) { return sh.ml[i]; },
        [&](int, int i) { return part + i * C::kPartPitch; });
    cluster.sync();  // a part stays until the cluster has read it
    return true;
}

// The pass with bf16 tiles after one with fp16 tiles that met a small group.
template <int D, int FMT>
__device__ __noinline__ void attend_small(const TreeParams &p, WideShared &sh, uint8_t *smem) {
    __syncthreads();  // all threads have left the first pass
    attend<D, FMT, false>(p, sh, smem);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) attn_tree_wide_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ WideShared sh;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr bool kHalf = FMT != SSA_KV_BF16;
    if (!attend<D, FMT, kHalf>(p, sh, smem) && kHalf) attend_small<D, FMT>(p, sh, smem);
}

template <int D, int FMT>
int launch(TreeParams &p, int rows, int entries, cudaStream_t s) {
    using C = Wide<D>;
    const int row_blocks = (rows + kM - 1) / kM;
    auto kernel = attn_tree_wide_kernel<D, FMT>;
    static std::atomic<uint64_t> done{0};  // devices whose limit is set
    int device = 0;
    SSA_CUDA_TRY(cudaGetDevice(&device));
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (!(done.load() & bit)) {
        SSA_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes));
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    // Slices of the list: as many as run at once, a tile each at least.
    static ClusterCounts clusters;
    p.slices = pick_slices(kernel, cfg, clusters, device, static_cast<long long>(p.B) * p.Hkv * row_blocks, (entries + kN - 1) / kN);
    cfg.gridDim = dim3(row_blocks * p.slices, p.Hkv, p.B);
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

template <int D>
int launch_format(TreeParams &p, int fmt, int rows, int entries, cudaStream_t s) {
    if (fmt == SSA_KV_BF16) return launch<D, SSA_KV_BF16>(p, rows, entries, s);
    if (fmt == SSA_KV_E4M3) return launch<D, SSA_KV_E4M3>(p, rows, entries, s);
    return launch<D, SSA_KV_E2M1>(p, rows, entries, s);
}

}  // namespace

int launch_tree_wide(TreeParams &p, int d, int fmt, int rows, int entries, cudaStream_t s) {
    return d == 64 ? launch_format<64>(p, fmt, rows, entries, s) : launch_format<128>(p, fmt, rows, entries, s);
}

}  // namespace ssa
