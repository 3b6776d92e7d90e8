"""Quantised caches whose groups are small (scale bytes below those of the fp16 products): the rows
of a layer with small values, of sinks with near-zero ones, of zeros.  Right within
test_gpu_tree's tolerances, and about as fast as any other rows.

A step with such a group is multiplied as bf16 with weights in two parts, twice the products of the
usual one; no kernel spends half its time on them, so twice the usual time bounds it (key by key
it was 6 to 240 times).  The kernel of many rows gives its pass up at the first such group and
takes the list again: where that is the last group of the list, the two passes are held to 2.5
times.  All-zero rows cost no more than small ones."""

import numpy as np
import pytest
import torch

import kv_ref as R
from gpu_util import dev, lists_to_device, t_i32
from test_gpu_tree import patterns, run, ssa

pytestmark = pytest.mark.gpu

ROWS_OF_FEW = [1, 4, 8, 16]  # nodes of 2 heads: up to 32 rows a KV head


def shifted(where, by, every=1):
    def edit(i, c, e):
        if "kv"[i] in where:
            e[:, :, ::every] = np.maximum(e[:, :, ::every].astype(int) - by, 16)
    return edit


def check_small(fmt, d, T, where, by, every, g=2):
    S = 400
    D, C = patterns(T + by, g, S, 200, 40)
    run(fmt, d, g, 1, S, T, [S - T, 250, 3], [T] * 3, D, C, 3, seed=T, edit=shifted(where, by, every))


@pytest.mark.parametrize("where,by,every", [("v", 9, 1), ("k", 20, 1), ("kv", 60, 1), ("kv", 14, 5), ("v", 200, 3)])
@pytest.mark.parametrize("T", ROWS_OF_FEW)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_small_groups_few_rows(fmt, d, T, where, by, every):
    check_small(fmt, d, T, where, by, every)


@pytest.mark.parametrize("where,by,every", [("v", 9, 1), ("k", 20, 1), ("kv", 60, 1), ("kv", 14, 5), ("v", 200, 3)])
@pytest.mark.parametrize("T,g", [(17, 2), (64, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_small_groups_many_rows(fmt, d, T, g, where, by, every):
    check_small(fmt, d, T, where, by, every, g)


def device_time(call):
    for _ in range(3):
        call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(4):
            call()
    best = float("inf")
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def time_ratio(fmt, d, T, edit):
    m = ssa()
    S, Hq, Hkv, B = 4096, 8, 2, 4
    D, C = [np.arange(700, dtype=np.int32)] * Hq, [np.arange(0, S, 9, dtype=np.int32)] * Hq
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), Hkv, depth=T)
    g = torch.Generator(device=dev()).manual_seed(3)
    rand = lambda *n: torch.randn(*n, device=dev(), generator=g).bfloat16()
    q, length = rand(B, T, Hq, d), t_i32([S - T] * B)
    cache = m.KVCache(B, Hkv, S, d, fmt, device=dev())
    m.kv_append(cache, rand(B * S, Hkv, d), rand(B * S, Hkv, d), t_i32([b * S for b in range(B + 1)]), t_i32([0] * B))
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out, lse = torch.empty_like(q), torch.empty(B, T, Hq, device=dev())
    call = lambda: m.attn_tree(q, cache, length, None, lists, out=out, lse=lse, status=status, check=False)
    usual = device_time(call)
    for i, (c, e) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        edit(i, c, e)
    small = device_time(call)
    assert int(status) == 0 and torch.isfinite(out).all()
    return small / usual


def smaller(where):  # by 2^16: below the fp16 range in either format
    def edit(i, c, e):
        if "kv"[i] in where:
            e -= 16
    return edit


def last_column(i, c, e):  # columns come behind the offsets in a list; 4023 is the last committed one for T = 64
    if i == 1:
        e[:, :, 4023] -= 16


def sinks(i, c, e):
    if i == 1:
        c[:, :, :4] = 0
        e[:, :, :4] = 16


def zeros(i, c, e):
    c.zero_()
    e.fill_(16)


@pytest.mark.parametrize("edit", [smaller("v"), smaller("kv"), sinks, zeros], ids=["values", "both", "sinks", "zeros"])
@pytest.mark.parametrize("T", [1, 4, 8])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_small_groups_are_as_fast_few_rows(fmt, T, edit):
    assert time_ratio(fmt, 128, T, edit) <= 2.0


@pytest.mark.parametrize("edit", [smaller("v"), smaller("kv"), sinks, zeros], ids=["values", "both", "sinks", "zeros"])
@pytest.mark.parametrize("T", [12, 64])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_small_groups_are_as_fast_many_rows(fmt, T, edit):
    assert time_ratio(fmt, 128, T, edit) <= 2.0


@pytest.mark.parametrize("T", [1, 8, 12, 64])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_a_small_group_at_the_end_of_a_list(fmt, T):
    assert time_ratio(fmt, 128, T, last_column) <= 2.5


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_waits_run_out_in_a_list_that_is_taken_again(fmt):
    # with the limit at 0 some wait of the first or of the second pass gives up; the same context
    # then runs a normal call
    m = ssa()
    S, T, d = 300, 40, 64
    D, C = patterns(51, 4, S, 150, 30)
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), 2, depth=T)
    g = torch.Generator(device=dev()).manual_seed(5)
    rand = lambda *n: torch.randn(*n, device=dev(), generator=g).bfloat16()
    cache = m.KVCache(2, 2, S, d, fmt, device=dev())
    m.kv_append(cache, rand(2 * S, 2, d), rand(2 * S, 2, d), t_i32([0, S, 2 * S]), t_i32([0, 0]))
    cache.v_scale[0] -= 16
    q, length = rand(2, T, 4, d), t_i32([200, 200])
    want = [x.clone() for x in m.attn_tree(q, cache, length, None, lists)]
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    old = m.set_wait_limit_ns(0)
    try:
        m.attn_tree(q, cache, length, None, lists, status=status, check=False)
        torch.cuda.synchronize()
    finally:
        m.set_wait_limit_ns(old)
    assert int(status) == -5
    for x, y in zip(m.attn_tree(q, cache, length, None, lists), want):
        assert torch.equal(x, y)


def test_a_list_taken_again_repeats_in_a_graph():
    # small groups in one of two sequences, other calls in flight on another stream
    m = ssa()
    S, T, d, Hq, Hkv = 2000, 40, 128, 8, 2
    D, C = [np.arange(700, dtype=np.int32)] * Hq, [np.arange(0, S, 17, dtype=np.int32)] * Hq
    lists = m.tree_lists(m.extend(*lists_to_device(D, C)[0], S), Hkv, depth=T)
    g = torch.Generator(device=dev()).manual_seed(6)
    rand = lambda *n: torch.randn(*n, device=dev(), generator=g).bfloat16()
    cache = m.KVCache(2, Hkv, S, d, "e4m3", device=dev())
    m.kv_append(cache, rand(2 * S, Hkv, d), rand(2 * S, Hkv, d), t_i32([0, S, 2 * S]), t_i32([0, 0]))
    cache.v_scale[1, :, 1000:] -= 16
    q, length = rand(2, T, Hq, d), t_i32([1900, 1900])
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    outs = [(torch.zeros_like(q), torch.zeros(2, T, Hq, device=dev())) for _ in range(3)]
    call = lambda o: m.attn_tree(q, cache, length, None, lists, out=o[0], lse=o[1], status=status, check=False)
    call(outs[0])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, o in zip(graphs, outs[1:]):
        with torch.cuda.graph(graph):
            call(o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert int(status) == 0 and outs[0][0].abs().sum() > 0
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
