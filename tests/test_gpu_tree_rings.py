"""GPU parity of sparse_attn_tree where one CTA walks a whole list: every ring of the kernels (rows
staged, entries resolved) wraps many times.

So many sequences run at once that no list is split over a cluster.  They are copies of three
sequences: those three are held against the fp64 reference within test_gpu_tree's tolerances, all
others have to repeat their bits."""

import numpy as np
import pytest
import torch

import kv_ref as R
from gpu_util import dev, lists_to_device, t_i32
from test_gpu_tree import check, make_cache, patterns, random_tree, run, ssa

pytestmark = pytest.mark.gpu

# copies of the three sequences with which no list is split: clusters of two CTAs would have to
# fit 378 times (148 SMs x 5 CTAs at most) or 114 times (one CTA an SM)
FEW, MANY = 126, 38


def run_copies(fmt, d, G, T, S, lengths, diags, verts, copies, depth=4, seed=0, edit=None, scale=None, q_edit=None):
    m = ssa()
    base, (kv, vv) = make_cache(fmt, 3, 1, S, d, seed, edit)
    many = lambda t: None if t is None else t.repeat(copies, *[1] * (t.dim() - 1))
    cache = m.KVCache.from_tensors(many(base.k), many(base.v), many(base.k_scale), many(base.v_scale), format=fmt)
    lists = m.tree_lists(m.extend(*lists_to_device(diags, verts)[0], S), 1, depth=depth)
    g = np.random.default_rng(seed + 7)
    q = R.bf16(g.standard_normal((3, T, G, d)))
    if q_edit:
        q_edit(q)
    par = random_tree(g, 3, T, depth)
    scale = d ** -0.5 if scale is None else scale
    tq = many(torch.from_numpy(q).to(dev()).bfloat16()).contiguous()
    O, L = m.attn_tree(tq, cache, many(t_i32(lengths)), many(t_i32(par)), lists, scale=scale)
    nodes = [T] * 3
    ref = R.tree_attention(q, kv, vv, lengths, par, nodes, diags, verts, scale, [0] * G)
    check(O[:3], L[:3], ref, nodes)
    bits = lambda x, t: x.view(t).view(copies, 3, *x.shape[1:])
    for x, t in ((O, torch.int16), (L, torch.int32)):
        y = bits(x, t)
        assert (y == y[:1]).all()
    return O[:3], L[:3]


def odd_groups(fmt, odd):
    """Groups that the products of whole tiles cannot take, in the keys `odd`: tiny, all-zero and
    (element 3's group of values) not finite in turn; for bf16 rows infinite values."""
    g = np.random.default_rng(11)

    def edit(i, c, e=None):
        if fmt == "bf16":
            if i == 1:
                c[:, :, odd, 3] = np.inf
            return
        e[:, :, odd[0::3]] = g.integers(60, 112, e[:, :, odd[0::3]].shape)
        e[:, :, odd[1::3]] = 16
        c[:, :, odd[1::3]] = 0
        if i == 1:
            c[:, :, odd[2::3], :32] = 0
            e[:, :, odd[2::3], 0] = 255
    return edit


# 8, 16 and 32 rows a KV head
@pytest.mark.parametrize("T", [4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_odd_groups_in_every_batch_of_a_long_list(fmt, d, T):
    # head 0 retains even columns and the node itself, head 1 everything; the first sequence's own
    # rows lie behind the odd ones, so its head 0 stays finite
    S, lengths = 1300, [1280, 1001, 700]
    D = [np.array([0], np.int32), np.arange(1250, dtype=np.int32)]
    C = [np.arange(0, S - 40, 2, dtype=np.int32), np.zeros(0, np.int32)]
    odd = np.arange(1, 1280, 6)
    O, L = run_copies(fmt, d, 2, T, S, lengths, D, C, FEW, edit=odd_groups(fmt, odd), seed=T)
    assert torch.isfinite(O[0, :, 0]).all() and torch.isfinite(L).all()
    assert torch.isfinite(O[:, :, 1, 32:]).all() and not torch.isfinite(O[:, :, 1, 3]).any()


# 40 and 128 rows a KV head, and two blocks of rows
@pytest.mark.parametrize("G,T", [(2, 20), (2, 64), (3, 50)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_odd_groups_in_every_tile_of_a_long_list(fmt, d, G, T):
    # lists of more than 17 tiles of 64 keys; heads as above, a third one like the second
    S, lengths = 1300, [1230, 1001, 700]
    D = [np.array([0], np.int32)] + [np.arange(1250, dtype=np.int32)] * (G - 1)
    C = [np.arange(0, S - 100, 2, dtype=np.int32)] + [np.zeros(0, np.int32)] * (G - 1)
    odd = np.arange(1, 1200, 48)
    O, L = run_copies(fmt, d, G, T, S, lengths, D, C, MANY, edit=odd_groups(fmt, odd), seed=T)
    assert torch.isfinite(O[0, :, 0]).all() and torch.isfinite(L).all()
    assert torch.isfinite(O[:, :, 1, 32:]).all() and not torch.isfinite(O[:, :, 1, 3]).any()


@pytest.mark.parametrize("T,copies", [(4, FEW), (8, FEW), (16, FEW), (20, MANY), (64, MANY)])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_many_light_keys_behind_a_heavy_one(fmt, T, copies):
    """The nearest key takes the weight 1 and has values of zero, over a thousand others weigh
    e^-17.8 = 2^-25.7 each with values of one: the output is their sum.  Weights that are rounded to
    fp16 are so against 2^7 or more for the largest: to half of 2^-24 that is 2^-32 of the largest a
    key, 1.3 % here; bf16 parts hold 16 bits of each."""
    m = ssa()
    S, d, ln = 1360, 64, 1280  # room for 64 nodes
    D, C = [np.arange(1, 1250, dtype=np.int32)] * 2, [np.zeros(0, np.int32)] * 2
    k, v = np.ones((1, 1, S, d)), np.ones((1, 1, S, d))
    k[..., 1::2] = -1
    k[:, :, ln - 1], v[:, :, ln - 1] = 2, 0
    v[:, :, ln - 1, ::32] = 1  # no group of zeros
    many = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev()).repeat(3 * copies, 1, 1, 1)
    if fmt == "bf16":
        cache = m.KVCache.from_tensors(many(k).bfloat16(), many(v).bfloat16())
    else:
        (kc, ks), (vc, vs) = R.encode(k, fmt), R.encode(v, fmt)
        assert (R.decode(kc, ks, fmt) == k).all() and (R.decode(vc, vs, fmt) == v).all()
        cache = m.KVCache.from_tensors(many(R.pack(kc, fmt)), many(R.pack(vc, fmt)), many(ks), many(vs), format=fmt)
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), 1, depth=1)
    q = torch.ones(3 * copies, T, 2, d, device=dev()).bfloat16()
    par = torch.full((3 * copies, T), -1, device=dev(), dtype=torch.int32)
    O, L = m.attn_tree(q, cache, torch.full((3 * copies,), ln, device=dev(), dtype=torch.int32), par, lists, scale=17.8 / 128)
    n, w = 1248, np.exp(-17.8)
    want = n * w / (1 + n * w)
    slack = 2.0 ** -8 * want + (n * 2.0 ** -32 if fmt != "bf16" else 2.0 ** -16 * want) + 2.0 ** -17 * want
    light = [e for e in range(d) if e % 32]
    err = (O[..., light].double() - want).abs().max().item()
    assert err <= slack, (err, slack)
    assert (L.double() - (17.8 + np.log1p(n * w))).abs().max().item() <= 1e-5


# every kernel at both head dimensions: 1 .. 8, 16 and 32 rows, blocks of 64 and 128 rows
@pytest.mark.parametrize("G,T", [(1, 1), (3, 5), (4, 4), (1, 17), (2, 16), (4, 8), (3, 11), (4, 16), (5, 13), (2, 64), (8, 16),
                                 (3, 43), (4, 64)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_row_counts_at_both_head_dimensions(fmt, d, G, T):
    S = 400
    D, C = patterns(G * 10 + T, 2 * G, S, 150, 40)
    run(fmt, d, 2 * G, 2, S, T, [S - T, 130], [T, max(1, T - 3)], D, C, max(1, T // 2), seed=T + 1)


# without odd groups: 4, 8, 16 and 32 rows, then 40, 128 and 150
@pytest.mark.parametrize("G,T", [(4, 1), (2, 4), (4, 4), (2, 16), (2, 20), (2, 64), (3, 50)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", R.FORMATS)
def test_long_lists_on_one_cta(fmt, d, G, T):
    S = 1300
    D = [np.arange(7 * h, 1150 + 7 * h, dtype=np.int32) for h in range(G)]
    C = [np.arange(h, S, 11, dtype=np.int32) for h in range(G)]
    run_copies(fmt, d, G, T, S, [1230, 1001, 700], D, C, FEW if G * T <= 32 else MANY, seed=T + G)


@pytest.mark.parametrize("G,T", [(2, 4), (2, 16), (2, 20), (3, 50)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_groups_that_are_not_finite_in_a_long_list(fmt, d, G, T):
    # among groups of ordinary size: the kernel of many rows stays with fp16 tiles
    S = 1300
    D = [np.array([0], np.int32)] + [np.arange(1250, dtype=np.int32)] * (G - 1)
    C = [np.arange(0, S - 100, 2, dtype=np.int32)] + [np.zeros(0, np.int32)] * (G - 1)
    odd = np.arange(1, 1200, 16)

    def edit(i, c, e):
        if i == 1:
            c[:, :, odd, :32] = 0
            e[:, :, odd, 0] = 255

    O, L = run_copies(fmt, d, G, T, S, [1230, 1001, 700], D, C, FEW if G * T <= 32 else MANY, edit=edit, seed=T)
    assert torch.isfinite(O[0, :, 0]).all() and torch.isfinite(L).all()
    assert torch.isfinite(O[:, :, 1, 32:]).all() and torch.isnan(O[:, :, 1, :32]).all()
