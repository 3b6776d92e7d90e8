"""GPU parity of sparse_attn_tree with the fp64 reference (kv_ref), and with the library's
own decoding and prefill.

Tolerances, derived before the first run: a logit's fp32 dot product of d terms is off by at
most ds = d 2^-23 scale sum|q_i k_i|; weights by a factor within 2 ds of 1 (numerator and
denominator), 2^-22 from the hardware's 2^x and 2^-12 from their rounding to fp16 (2^-25 absolutely
where they are under 2^-14; the largest is at least 1, so against the sum at most
2^-25 a key), so |O - ref| <= (2 ds + 2^-11) sum p|v| + keys 2^-25 max|v| before the rounding to bf16 (half a step, 2^-8 |O|),
and |LSE - ref| <= ds + 2^-20 (1 + |LSE|).
"""

import subprocess
import sys

import numpy as np
import pytest
import torch

import kv_ref as R
from conftest import ROOT
from gpu_util import dev, lists_to_device, t_i32
from structured_sparse_attention_b200 import inputs

pytestmark = pytest.mark.gpu


def ssa():
    import structured_sparse_attention_b200 as m
    return m


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def random_tree(g, B, T, depth):
    parent = np.full((B, T), -1, np.int32)
    for b in range(B):
        t = np.zeros(T, int)
        for n in range(1, T):
            p = int(g.integers(-1, n))
            if p >= 0 and t[p] + 1 >= depth:
                p = -1
            parent[b, n], t[n] = p, (t[p] + 1 if p >= 0 else 0)
    return parent


def make_cache(fmt, B, Hkv, S, d, seed, edit=None):
    """A cache of random rows, and its values in fp64."""
    m = ssa()
    g = np.random.default_rng(seed)
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev())
    parts, vals = [], []
    for i in range(2):
        x = R.bf16(g.standard_normal((B, Hkv, S, d)))
        if fmt == "bf16":
            if edit:
                edit(i, x)
            parts.append(T(x).bfloat16())
            vals.append(x)
        else:
            c, e = R.encode(x, fmt)
            if edit:
                edit(i, c, e)
            parts.append((T(R.pack(c, fmt)), T(e)))
            vals.append(R.decode(c, e, fmt))
    if fmt == "bf16":
        return m.KVCache.from_tensors(*parts, format=fmt), vals
    (k, ks), (v, vs) = parts
    return m.KVCache.from_tensors(k, v, ks, vs, format=fmt), vals


def check(O, LSE, ref, nodes):
    o, l = f64(O), LSE.cpu().numpy().astype(np.float64)
    Or, Lr, eo, el = ref
    for b, nn in enumerate(nodes):
        nn = int(nn)
        x, y = o[b, :nn], Or[b, :nn]
        fin = np.isfinite(y)
        assert (np.isnan(x) == np.isnan(y)).all() and (x[np.isinf(y)] == y[np.isinf(y)]).all()
        err = np.abs(x - y)[fin] - (2.0 ** -8 * np.abs(y) + 1.01 * eo[b, :nn])[fin]
        assert (err <= 0).all(), float(err.max())
        u, w = l[b, :nn], Lr[b, :nn]
        fin = np.isfinite(w)
        assert (np.isneginf(u) == np.isneginf(w)).all() and (np.isnan(u) == np.isnan(w)).all()
        assert (np.abs(u - w)[fin] <= el[b, :nn][fin]).all(), float((np.abs(u - w) - el[b, :nn])[fin].max())
        assert (x[np.isneginf(w)] == 0).all()


def run(fmt, d, Hq, Hkv, S, T, length, nodes, diags, verts, depth, parent="random", seed=0, kv_map=None, edit=None,
        scale=None, q_edit=None, slack=0, lists_depth=None):
    m = ssa()
    B = len(length)
    g = np.random.default_rng(seed + 99)
    cache, (kv, vv) = make_cache(fmt, B, Hkv, S, d, seed, edit)
    dl, _ = lists_to_device(diags, verts)
    plan = m.extend(*dl, S)
    km = None if kv_map is None else t_i32(kv_map)
    lists = m.tree_lists(plan, Hkv, depth=lists_depth or depth, kv_map=km)
    q = R.bf16(g.standard_normal((B, T, Hq, d)))
    if q_edit:
        q_edit(q)
    par = random_tree(g, B, T, depth) if isinstance(parent, str) else parent
    tq = torch.from_numpy(q).to(dev()).bfloat16()
    out = torch.full((B, T, Hq, d), 5.0, device=dev(), dtype=torch.bfloat16)
    lse = torch.full((B, T, Hq), 5.0, device=dev())
    scale = d ** -0.5 if scale is None else scale
    O, L = m.attn_tree(tq, cache, t_i32(length), None if par is None else t_i32(par), lists, n_nodes=t_i32(nodes),
                       scale=scale, out=out, lse=lse)
    pr = np.tile(np.arange(T) - 1, (B, 1)) if par is None else par
    kvh = kv_map if kv_map is not None else np.arange(Hq) // (Hq // Hkv)
    ref = R.tree_attention(q, kv, vv, length, pr, nodes, diags, verts, scale, kvh)
    check(O, L, ref, nodes)
    for b, nn in enumerate(nodes):  # rows behind the last node are left as they were
        assert (O[b, int(nn):] == 5).all() and (L[b, int(nn):] == 5).all()
    return O, L, (tq, cache, lists, plan)


def patterns(seed, H, S, nd=60, nc=20):
    return inputs.random_patterns(seed, H, S, min(nd, S), min(nc, S))


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_single_token(fmt, d):
    S = 700
    D, C = patterns(1, 8, S, 300, 60)
    run(fmt, d, 8, 2, S, 1, [0, 1, 300, 699], [1] * 4, D, C, 1)


# rows per KV head: 1 .. 16 go one way, then blocks of 32, 64 and 128 rows
@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("G,T", [(1, 1), (3, 5), (4, 4), (1, 17), (2, 16), (4, 8), (3, 11), (4, 16), (5, 13), (2, 64),
                                 (8, 16), (3, 43), (4, 64)])
def test_row_counts(fmt, G, T):
    S, d = 400, 128 if (G + T) % 2 else 64
    D, C = patterns(G * 100 + T, 2 * G, S, 150, 40)
    run(fmt, d, 2 * G, 2, S, T, [S - T, 130], [T, max(1, T - 3)], D, C, max(1, T // 2), seed=T)


@pytest.mark.parametrize("fmt,T", [("bf16", 1), ("e4m3", 4), ("e2m1", 30), ("bf16", 40), ("e4m3", 64)])
def test_long_lists_over_several_slices(fmt, T):
    # 1500 keys a KV head: 8 CTAs share a list
    S = 4000
    D = [np.arange(20 * h, 20 * h + 1200, dtype=np.int32) for h in range(4)]
    C = [np.arange(h, S, 13, dtype=np.int32) for h in range(4)]
    run(fmt, 128, 4, 2, S, T, [3900], [T], D, C, 3, seed=5)


def test_lists_longer_than_a_chunk_on_one_cta():
    # many sequences: one CTA walks a whole list of over 256 keys
    S = 900
    D = [np.arange(500, dtype=np.int32)] * 2
    C = [np.arange(5, 880, 7, dtype=np.int32)] * 2
    B = 160
    for fmt, T in (("e4m3", 1), ("e2m1", 20)):
        run(fmt, 64, 2, 2, S, T, list(np.linspace(0, S - T, B).astype(int)), [T] * B, D, C, 2, seed=8)


@pytest.mark.parametrize("T", [1, 7, 33])
def test_rows_that_retain_nothing(T):
    # the nearest diagonal is 50 away: nodes of short sequences have no key at all
    D, C = [np.array([50, 90], np.int32)] * 2, [np.array([200], np.int32), np.zeros(0, np.int32)]
    O, L, _ = run("e4m3", 64, 2, 1, 256, T, [0, 20, 49, 50, 201], [T] * 5, D, C, 1)
    assert torch.isneginf(L[0]).all() and (O[0] == 0).all()


@pytest.mark.parametrize("T", [1, 6, 40])
def test_no_pattern_at_all(T):
    Z = [np.zeros(0, np.int32)] * 2
    O, L, _ = run("bf16", 128, 2, 2, 100, T, [60], [T], Z, Z, 2)
    assert torch.isneginf(L).all() and (O == 0).all()


def test_chain_and_explicit_parents_agree():
    D, C = patterns(5, 4, 300)
    T = 9
    O, L, _ = run("e2m1", 64, 4, 2, 300, T, [100, 291], [T, T], D, C, T, parent=None)
    par = np.tile(np.arange(T, dtype=np.int32) - 1, (2, 1))
    O2, L2, _ = run("e2m1", 64, 4, 2, 300, T, [100, 291], [T, T], D, C, T, parent=par)
    assert torch.equal(O, O2) and torch.equal(L, L2)


def test_deep_chain_of_64():
    D, C = patterns(6, 4, 300, 100, 30)
    run("bf16", 64, 4, 2, 300, 64, [236, 0], [64, 63], D, C, 64, parent=None)


def test_lists_deeper_than_the_trees():
    D, C = patterns(7, 4, 500, 40, 30)
    run("e4m3", 128, 4, 2, 500, 12, [400, 123], [12, 5], D, C, 3, lists_depth=64)


def test_explicit_kv_map_with_uneven_groups():
    D, C = patterns(8, 7, 300)
    for T in (1, 3, 20):
        run("e4m3", 64, 7, 3, 300, T, [250, 17], [T, T], D, C, 2, kv_map=np.array([2, 0, 2, 2, 0, 2, 2], np.int32))


def test_ragged_node_counts_include_none():
    D, C = patterns(9, 6, 300)
    run("e2m1", 128, 6, 2, 300, 10, [250, 90, 290, 0], [10, 0, 3, 7], D, C, 4)


def test_window_offsets_at_word_ends():
    # diagonals around multiples of 64 and depths that carry across them
    D = [np.array([0, 1, 62, 63, 64, 65, 127, 128, 191, 192, 255, 299], np.int32)] * 2
    run("bf16", 64, 2, 1, 300, 30, [236, 256, 192, 64, 63], [30] * 5, D, [np.array([63, 64, 128], np.int32)] * 2, 30)


@pytest.mark.parametrize("T", [1, 5, 20, 40])
def test_values_outside_a_rows_keys_do_not_touch_it(T):
    # NaN and infinite keys and values: rows that do not retain them stay finite, and rows
    # behind the last node (never written, here NaN) are not read
    S, ln = 200, 150
    D = [np.array([0, 1, 2, 3], np.int32), np.arange(0, 60, dtype=np.int32)]
    C = [np.array([5, 90], np.int32), np.array([7], np.int32)]

    def edit(i, x):
        x[:, :, 7] = np.nan                 # head 1 only
        if i == 1:
            x[:, :, 120] = np.inf           # head 1 only
            x[:, :, 90, :3] = -np.inf       # head 0 only
        else:
            x[:, :, 120] = 0.25
        x[:, :, ln + T:] = np.nan
        x[:, :, 30] = np.nan                # nobody

    O, L, _ = run("bf16", 64, 2, 1, S, T, [ln], [T], D, C, 1, parent=np.full((1, T), -1, np.int32), edit=edit)
    assert torch.isfinite(O[:, :, 0, 3:]).all() and torch.isfinite(L[:, :, 0]).all()
    assert torch.isneginf(O[:, :, 0, :3]).all() and torch.isnan(O[:, :, 1]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T", [1, 4, 33])
@pytest.mark.parametrize("where", ["k", "v", "both"])
def test_scales_of_every_size(fmt, T, where):
    # groups of zeros, tiny and huge ones among ordinary keys, and queries of any size
    D, C = patterns(17, 4, 200, 60, 20)
    g = np.random.default_rng(3)

    def edit(i, c, e):
        if where in ("both", "kv"[i]):
            e[:, :, ::3] = np.where(g.random(e[:, :, ::3].shape) < 0.5, e[:, :, ::3], g.integers(60, 118, e[:, :, ::3].shape))
            e[:, :, 5::17] = 16
            c[:, :, 5::17] = 0
            if i == 1:
                e[:, :, 7::19] = 134 if fmt == "e4m3" else 140

    def q_edit(q):
        q[:, :, 1] *= 2.0 ** -60
        q[:, :, 2] *= 2.0 ** 3
        q[:, :, 3] = 0
    run(fmt, 64, 4, 2, 200, T, [150, 60], [T, T], D, C, 2, edit=edit, q_edit=q_edit)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T", [2, 33])
def test_nan_groups_of_a_quantised_cache(fmt, T):
    D, C = [np.arange(3, dtype=np.int32), np.arange(40, dtype=np.int32)], [np.zeros(0, np.int32)] * 2

    def edit(i, c, e):
        if i == 1:
            c[:, :, 80, 32:64] = 0
            e[:, :, 80, 1] = 255

    O, L, _ = run(fmt, 128, 2, 1, 160, T, [100], [T], D, C, 1, parent=np.full((1, T), -1, np.int32), edit=edit)
    assert torch.isfinite(O[:, :, 0]).all() and torch.isnan(O[:, :, 1, 32:64]).all()
    assert torch.isfinite(O[:, :, 1, :32]).all() and torch.isfinite(O[:, :, 1, 64:]).all()


def test_infinite_logits():
    def q_edit(q):
        q[0, 0, 0] = np.inf
        q[0, 1, 1, 0] = np.nan
    D, C = [np.arange(30, dtype=np.int32)] * 2, [np.zeros(0, np.int32)] * 2
    m = ssa()
    for T in (2, 20):
        q = torch.randn(1, T, 2, 64, device=dev()).bfloat16()
        q[0, 0, 0], q[0, 1, 1, 0] = float("inf"), float("nan")
        cache, (kv, vv) = make_cache("bf16", 1, 1, 100, 64, 3)
        plan = m.extend(*lists_to_device(D, C)[0], 100)
        par = np.full((1, T), -1, np.int32)
        O, L = m.attn_tree(q, cache, t_i32([50]), t_i32(par), m.tree_lists(plan, 1))
        assert torch.isnan(O[0, 0, 0]).all() and torch.isnan(O[0, 1, 1]).all()
        ok = torch.ones(T, 2, dtype=torch.bool, device=dev())
        ok[0, 0] = ok[1, 1] = False
        assert torch.isfinite(O[0][ok]).all() and torch.isfinite(L[0][ok]).all()


def test_large_logits_keep_their_maximum():
    D, C = patterns(12, 2, 300, 100, 20)
    for T in (2, 30):
        run("bf16", 64, 2, 1, 300, T, [260], [T], D, C, 2, scale=40.0)


def test_nodes_agree_with_decoding_after_their_path_is_committed():
    # bf16 cache: node n's row is sparse_attn_decode's once the path lies in rows len, len + 1, ...
    m = ssa()
    S, d, Hq, Hkv, T = 300, 64, 4, 2, 12
    D, C = patterns(13, Hq, S, 120, 40)
    ln = 200
    g = np.random.default_rng(0)
    par = random_tree(g, 1, T, 5)
    O, L, (q, cache, lists, plan) = run("bf16", d, Hq, Hkv, S, T, [ln], [T], D, C, 5, parent=par, seed=21)
    for n, path in enumerate(R.tree_paths(par[0], T)):
        k, v = cache.k.clone(), cache.v.clone()
        for t, a in enumerate(path):
            k[:, :, ln + t], v[:, :, ln + t] = cache.k[:, :, ln + a], cache.v[:, :, ln + a]
        o, l = m.attn_decode(q[:, n], k, v, t_i32([ln + len(path) - 1]), plan)
        assert torch.allclose(l, L[:, n], atol=2e-4)
        assert torch.allclose(o.float(), O[:, n].float(), atol=2e-2)


def test_rows_past_32_bits():
    m = ssa()
    B, H, S, d = 2, 16, 600000, 128
    cache = m.KVCache(B, H, S, d, "bf16", device=dev())
    D = [np.arange(40, dtype=np.int32)] * H
    C = [np.array([0, 599000], np.int32)] * H
    plan = m.extend(*lists_to_device(D, C)[0], S)
    ln = S - 2
    rows = sorted({0, 599000} | set(range(ln - 45, S)))
    cache.k[1][:, rows] = torch.randn(H, len(rows), d, device=dev()).bfloat16()
    cache.v[1][:, rows] = torch.randn(H, len(rows), d, device=dev()).bfloat16()
    q = torch.randn(B, 2, H, d, device=dev()).bfloat16()
    O, L = m.attn_tree(q, cache, t_i32([1, ln]), None, m.tree_lists(plan, H, depth=2))
    o, l = m.attn_decode(q[:, 1].contiguous(), cache.k, cache.v, t_i32([2, ln + 1]), plan)
    assert torch.allclose(l, L[:, 1], atol=2e-4) and torch.allclose(o.float(), O[:, 1].float(), atol=2e-2)


@pytest.mark.parametrize("what", ["length", "long", "count", "parent", "self", "deep"])
def test_bad_sequences_are_reported_and_empty(what):
    m = ssa()
    S, T = 64, 4
    D, C = [np.arange(20, dtype=np.int32)] * 2, [np.zeros(0, np.int32)] * 2
    cache, _ = make_cache("e4m3", 2, 1, S, 64, 1)
    plan = m.extend(*lists_to_device(D, C)[0], S)
    lists = m.tree_lists(plan, 1, depth=2)
    length, nodes, par = [30, 30], [4, 4], np.array([[-1, 0, 0, -1]] * 2, np.int32)
    if what == "length":
        length[1] = -1
    elif what == "long":
        length[1] = S - 3
    elif what == "count":
        nodes[1] = 5
    elif what == "parent":
        par[1, 2] = -2
    elif what == "self":
        par[1, 2] = 2
    else:
        par[1, 2] = 1
    q = torch.randn(2, T, 2, 64, device=dev()).bfloat16()
    out, lse = torch.full_like(q, 3.0), torch.full((2, T, 2), 3.0, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    m.attn_tree(q, cache, t_i32(length), t_i32(par), lists, n_nodes=t_i32(nodes), out=out, lse=lse, status=status, check=False)
    torch.cuda.synchronize()
    assert int(status) == -1
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert torch.isfinite(lse[0]).all() and (out[0] != 3).any()
    with pytest.raises(m.SSAError):
        m.attn_tree(q, cache, t_i32(length), t_i32(par), lists, n_nodes=t_i32(nodes))


def test_lists_are_the_unions():
    m = ssa()
    S, H, Hkv = 333, 6, 2
    D, C = patterns(31, H, S, 80, 30)
    plan = m.extend(*lists_to_device(D, C)[0], S)
    for depth in (1, 2, 3, 33, 64):
        t = m.tree_lists(plan, Hkv, depth=depth)
        op, cp = t.off_ptr.tolist(), t.col_ptr.tolist()
        for g in range(Hkv):
            heads = range(3 * g, 3 * g + 3)
            want = sorted({int(r) - k for h in heads for r in D[h] for k in range(depth)} - set(range(-64, 1)))
            offs, cols = t.offs[op[g]:op[g + 1]].tolist(), t.cols[cp[g]:cp[g + 1]].tolist()
            assert [o for o, _ in offs] == want
            assert [c for c, _ in cols] == sorted({int(c) for h in heads for c in C[h]})
            sets = [set(D[h].tolist()) for h in heads]
            for o, bits in offs[::5]:
                hits = [sum(o + k in d for k in range(depth)) for d in sets]
                assert bits == sum((n == depth) << i | (n > 0) << (16 + i) for i, n in enumerate(hits))
            for c, bits in cols:
                assert bits == sum(0x10001 << i for i, h in enumerate(heads) if c in C[h])
            for w in range(t.sizes.words):
                assert int(t.off_rank[g, w]) == sum(o < 64 * w for o in want)
                assert int(t.col_rank[g, w]) == sum(c < 64 * w for c, _ in cols)
        assert t.sizes.max_entries == max(op[g + 1] - op[g] + cp[g + 1] - cp[g] for g in range(Hkv))


def test_bad_kv_map_is_refused():
    m = ssa()
    D, C = patterns(2, 4, 50)
    plan = m.extend(*lists_to_device(D, C)[0], 50)
    with pytest.raises(m.SSAError):
        m.tree_lists(plan, 2, kv_map=t_i32([0, 1, 2, 0]))


def test_captured_replayed_and_deterministic():
    # two graphs and an eager call on another stream give the same bits
    m = ssa()
    S, T, Hq, Hkv, d = 2000, 6, 8, 2, 128
    D, C = [np.arange(700, dtype=np.int32)] * Hq, [np.arange(0, S, 17, dtype=np.int32)] * Hq
    cache, _ = make_cache("e4m3", 2, Hkv, S, d, 4)
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), Hkv, depth=6)
    q = torch.randn(2, T, Hq, d, device=dev()).bfloat16()
    length = t_i32([1900, 800])
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    outs = [(torch.zeros_like(q), torch.zeros(2, T, Hq, device=dev())) for _ in range(3)]
    call = lambda o, **kw: m.attn_tree(q, cache, length, None, lists, out=o[0], lse=o[1], status=status, check=False, **kw)
    call(outs[0])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr, o in zip(graphs, outs[1:]):
        with torch.cuda.graph(gr):
            call(o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
    length.copy_(t_i32([1000, 1994]))  # read at replay
    graphs[0].replay()
    call(outs[0], stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(outs[1][0], outs[0][0]) and int(status) == 0


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_prefill_draft_verify_commit(fmt):
    """The operators as a serving loop uses them: append a prompt, run the prefill attention on
    the values as stored, append a drafted tree and attend to it, commit one path by
    appending it again, and decode the next token: each step matches the reference."""
    m = ssa()
    d, Hq, Hkv, S, n, T = 64, 4, 2, 256, 200, 7
    D, C = patterns(41, Hq, S, 90, 30)
    (dl, host), seed = lists_to_device(D, C), 5
    plan = m.extend(*dl, S)
    lists = m.tree_lists(plan, Hkv, depth=4)
    freqs = 10000.0 ** (-np.arange(d // 2) * 2.0 / d)
    w = 1 + 0.1 * np.random.default_rng(1).standard_normal(d).astype(np.float32)
    tf, tw = torch.from_numpy(freqs).to(dev()), torch.from_numpy(w).to(dev())
    gen = torch.Generator(device=dev())
    gen.manual_seed(seed)
    proj = lambda k: torch.randn(k, Hq + 2 * Hkv, d, device=dev(), generator=gen).bfloat16()
    cut = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
    cache = m.KVCache(1, Hkv, S, d, fmt, device=dev())

    def append(x, row0, pos=None, queries=True, **kw):
        q, k, v = cut(x)
        return m.kv_append(cache, k, v, t_i32([0, len(x)]), t_i32([row0]), q=q if queries else None,
                           pos=None if pos is None else t_i32(pos), freqs=tf, q_weight=tw if queries else None, k_weight=tw, **kw)

    # prompt: stored values come back head-major for the prefill attention
    x = proj(n)
    heads = lambda h: torch.zeros(h, S, d, device=dev(), dtype=torch.bfloat16)
    qp, kp, vp = heads(Hq), heads(Hkv), heads(Hkv)
    at = lambda t: t[:, :n].transpose(0, 1)
    append(x, 0, q_out=at(qp), k_out=at(kp), v_out=at(vp))
    k2, v2 = m.kv_read(cache, t_i32([0, n]), t_i32([0]), n)
    assert torch.equal(k2, at(kp)) and torch.equal(v2, at(vp))
    O, L = m.attn_fwd(qp, kp, vp, plan)
    # the last prompt token again, as a tree of one node over n - 1 rows
    o1, l1 = m.attn_tree(qp[:, n - 1][None, None].contiguous(), cache, t_i32([n - 1]), None, lists)
    assert torch.allclose(L[:, n - 1], l1[0, 0], atol=1e-3) and torch.allclose(O[:, n - 1].float(), o1[0, 0].float(), atol=2e-2)

    # a tree of T nodes
    par = np.array([[-1, 0, 0, 1, 1, 3, -1]], np.int32)
    paths = R.tree_paths(par[0], T)
    pos = [n + len(p) - 1 for p in paths]
    y = proj(T)
    qt = append(y, n, pos)
    ot, lt = m.attn_tree(qt[None], cache, t_i32([n]), t_i32(par), lists)
    kv = [f64(t).transpose(1, 0, 2)[None] for t in m.kv_read(cache, t_i32([0, n + T]), t_i32([0]), n + T)]
    pad = lambda a: np.concatenate([a, np.zeros((1, Hkv, S - n - T, d))], 2)
    ref = R.tree_attention(f64(qt)[None], pad(kv[0]), pad(kv[1]), [n], par, [T], D, C, d ** -0.5, np.arange(Hq) // 2)
    check(ot, lt, ref, [T])

    # the path 0, 1, 3, 5 is accepted: its tokens again, at their final rows
    path = paths[5]
    append(y[path].contiguous(), n, queries=False)
    z = proj(1)
    qz = append(z, n + 4)
    oz, lz = m.attn_tree(qz[None], cache, t_i32([n + 4]), None, lists)
    k, v = (f64(t).transpose(1, 0, 2)[None] for t in m.kv_read(cache, t_i32([0, n + 5]), t_i32([0]), n + 5))
    np.testing.assert_array_equal(k[0, :, n:n + 4], kv[0][0, :, [n + a for a in path]].transpose(1, 0, 2))
    full = np.zeros((2, 1, Hkv, S, d))
    full[0, :, :, :n + 5], full[1, :, :, :n + 5] = k, v
    ref = R.tree_attention(f64(qz)[None], full[0], full[1], [n + 4], [[-1]], [1], D, C, d ** -0.5, np.arange(Hq) // 2)
    check(oz, lz, ref, [1])
    if fmt == "bf16":  # and the framework's own decoding step on the same cache
        od, ld = m.attn_decode(qz, cache.k, cache.v, t_i32([n + 4]), plan)
        assert torch.allclose(ld, lz[:, 0], atol=2e-4) and torch.allclose(od.float(), oz[:, 0].float(), atol=2e-2)


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_wait_expiry_returns_timeout_then_recovers(fmt):
    # trees of many rows wait on barriers inside the kernel; with the limit at 0 the first wait
    # that is not complete gives up, and the same context then runs a normal call
    m = ssa()
    S, T, d = 300, 40, 64
    D, C = patterns(51, 4, S, 150, 30)
    cache, _ = make_cache(fmt, 1, 2, S, d, 1)
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), 2, depth=T)
    q = torch.randn(1, T, 4, d, device=dev()).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    old = m.set_wait_limit_ns(0)
    try:
        m.attn_tree(q, cache, t_i32([200]), None, lists, status=status, check=False)
        torch.cuda.synchronize()
    finally:
        m.set_wait_limit_ns(old)
    assert int(status) == -5
    run(fmt, d, 4, 2, S, T, [200], [T], D, C, T, parent=None)


def test_batches_of_many_heads_without_marks():
    # more than 16 query heads on one KV head: the lists carry no marks for the rest
    S, H = 200, 20
    D, C = patterns(61, H, S, 60, 20)
    for T in (1, 2, 5):
        run("e4m3", 64, H, 1, S, T, [150, 195], [T, T], D, C, T)


def test_a_lone_sequence_shorter_than_a_step():
    D, C = patterns(62, 4, 40, 30, 10)
    for T in (1, 9, 20):
        run("e2m1", 128, 4, 2, 40, T, [3], [T], D, C, 3)


@pytest.mark.parametrize("what", ["length", "far below", "far above", "count", "parent", "deep"])
@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("T", [4, 40])
def test_sequences_far_out_of_range_are_reported_and_empty(T, fmt, what):
    """Both kernels read ahead in the lists; of a bad sequence they read none."""
    m = ssa()
    S = 256
    D, C = [np.arange(200, dtype=np.int32)] * 2, [np.arange(0, 256, 3, dtype=np.int32)] * 2
    cache, _ = make_cache(fmt, 2, 1, S, 64, 1)
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), 1, depth=2)
    length, nodes, par = [100, 100], [T, T], np.array([[-1] + [0] * (T - 1)] * 2, np.int32)
    if what == "length":
        length[1] = -1
    elif what == "far below":
        length[1] = -(2**31)
    elif what == "far above":
        length[1] = 2**31 - 1
    elif what == "count":
        nodes[1] = T + 1
    elif what == "parent":
        par[1, 2] = 2
    else:
        par[1, 2] = 1
    q = torch.randn(2, T, 2, 64, device=dev()).bfloat16()
    out, lse = torch.full_like(q, 3.0), torch.full((2, T, 2), 3.0, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    m.attn_tree(q, cache, t_i32(length), t_i32(par), lists, n_nodes=t_i32(nodes), out=out, lse=lse, status=status, check=False)
    torch.cuda.synchronize()
    assert int(status) == -1
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert torch.isfinite(lse[0]).all() and (out[0] != 3).any()


def test_calls_at_once_on_several_streams():
    """Both kernels of the tree attention, an append to another cache and the prefill attention (which
    holds tensor memory too) run side by side and give the bits that each gives alone."""
    m = ssa()
    S, Hq, Hkv, d = 4096, 8, 2, 128
    D, C = [np.arange(900, dtype=np.int32)] * Hq, [np.arange(0, S, 19, dtype=np.int32)] * Hq
    plan = m.extend(*lists_to_device(D, C)[0], S)
    g = torch.Generator(device=dev()).manual_seed(7)
    rand = lambda *n: torch.randn(*n, device=dev(), generator=g).bfloat16()
    caches = [make_cache(fmt, 6, Hkv, S, d, 5)[0] for fmt in ("e4m3", "bf16")]
    lists = m.tree_lists(plan, Hkv, depth=64)
    length = t_i32([S - 64, 100, 2000, 3000, 900, 0])
    narrow, wide = rand(6, 5, Hq, d), rand(6, 64, Hq, d)
    q, k, v = rand(Hq, S, d), rand(Hkv, S, d), rand(Hkv, S, d)
    other = m.KVCache(1, Hkv, S, d, "e2m1")
    kt, vt = k.transpose(0, 1), v.transpose(0, 1)
    ptr, row0 = t_i32([0, S]), t_i32([0])
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    kw = dict(check=False, status=status)

    work = [lambda: m.attn_tree(narrow, caches[0], length, None, lists, **kw),
            lambda: m.attn_tree(wide, caches[0], length, None, lists, **kw),
            lambda: m.attn_tree(wide, caches[1], length, None, lists, **kw),
            lambda: m.attn_fwd(q, k, v, plan, check=False),
            lambda: (m.kv_append(other, kt, vt, ptr, row0, **kw), other.k, other.k_scale)[1:]]
    alone = [[x.clone() for x in call()] for call in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in alone]
    results = []
    for _ in range(4):
        for call, stream in zip(work, streams):
            with torch.cuda.stream(stream):
                results.append(call())
    torch.cuda.synchronize()
    assert int(status) == 0
    for i, got in enumerate(results):
        for x, y in zip(got, alone[i % len(alone)]):
            assert torch.equal(x, y), i


FIRST_CALLS = """
import numpy as np, torch
import structured_sparse_attention_b200 as m
dev = torch.device("cuda:0")
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
S, H, d = 1024, 4, 128
plan = m.extend(i32([0, 300, 600, 900, 1200]), i32(list(range(300)) * 4), i32([0, 2, 4, 6, 8]), i32([0, 5] * 4), S)
lists = m.tree_lists(plan, 1, depth=20)
cache = m.KVCache(1, 1, S, d, "e4m3")
k = torch.randn(S, 1, d, device=dev).bfloat16()
status = torch.zeros(1, dtype=torch.int32, device=dev)
qs = [torch.randn(1, T, H, d, device=dev).bfloat16() for T in (1, 20)]
outs = [(torch.zeros_like(q), torch.zeros(q.shape[:3], device=dev)) for q in qs]
ptr, row0, length = i32([0, S]), i32([0]), i32([S - 20])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def step(out):
    m.kv_append(cache, k, k, ptr, row0, check=False, status=status)
    for q, (o, l) in zip(qs, out):
        m.attn_tree(q, cache, length, None, lists, out=o, lse=l, check=False, status=status)
with torch.cuda.graph(graph):
    step(outs)
graph.replay()
torch.cuda.synchronize()
again = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in outs]
step(again)
torch.cuda.synchronize()
assert int(status) == 0 and all(torch.equal(a, b) and a.abs().sum() > 0 for x, y in zip(outs, again) for a, b in zip(x, y))
print("ok")
"""


def test_first_calls_of_a_process_inside_a_capture():
    # what a launch asks of the device once (limits, clusters that fit) is asked while capturing
    out = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip().endswith("ok"), out.stderr[-2000:]


@pytest.mark.parametrize("T", [2, 9, 33])
@pytest.mark.parametrize("fmt,top", [("e4m3", 134), ("e2m1", 140)])
def test_scale_bytes_out_of_range_are_reported(fmt, top, T):
    # only of rows that the call reads; the other sequence's result is what it was
    m = ssa()
    S, d = 300, 128
    D, C = [np.array([0, 3, 5], np.int32)] * 2, [np.array([11], np.int32)] * 2
    cache, _ = make_cache(fmt, 2, 1, S, d, 1)
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), 1, depth=1)
    q = torch.randn(2, T, 2, d, device=dev()).bfloat16()
    par, length = t_i32(np.full((2, T), -1, np.int32)), t_i32([150, 200])
    call = lambda: m.attn_tree(q, cache, length, par, lists)
    O, L = (x.clone() for x in call())
    for t in (cache.k_scale, cache.v_scale):
        keep = t.clone()
        t[0, 0, 50] = top + 1  # nobody's
        o, l = call()
        assert torch.equal(o, O) and torch.equal(l, L)
        for row, E in ((147, top + 1), (11, 142), (150, 254)):
            t[0, 0, row, 2] = E
            status = torch.zeros(1, dtype=torch.int32, device=dev())
            o, l = m.attn_tree(q, cache, length, par, lists, status=status, check=False)
            assert int(status) == -1 and torch.equal(o[1], O[1]) and torch.equal(l[1], L[1])
            t.copy_(keep)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("T", [2, 9, 40])
def test_the_smallest_scales(fmt, T):
    # scales whose product with a row's shift is below fp32: all logits are zero, masks still hold,
    # and so do small groups
    D, C = patterns(71, 2, 300, 60, 20)

    def q_edit(q):
        q[:, 0] *= 2.0 ** -60
        q[:, 1] = 0

    def edit(i, c, e=None):
        if e is not None:
            e[:, :, 200::40] = 100

    for scale in (1e-37, 2.0 ** -100):
        run(fmt, 64, 2, 1, 300, T, [250, 130], [T, T], D, C, 2, q_edit=q_edit, edit=edit, scale=scale)
