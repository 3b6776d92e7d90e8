"""GPU parity of sparse_kv_append and sparse_kv_read with the fp64 reference (kv_ref).

Tolerances, derived before the first run:
* values that are stored as they come (V) and everything read back are exact;
* a normalised, rotated element goes through a sum of d squares, a reciprocal square root,
  two products, one rotation and the angle's sine and cosine, all fp32: under 30 roundings
  of 2^-24 of its pair's magnitude, so |y - ref| <= 2^-19 |pair| before the last rounding;
* the last rounding is half a step: 2^-8 |y| for bf16, half the code spacing for codes.
"""

import numpy as np
import pytest
import torch

import kv_ref as R
from gpu_util import dev, t_i32
from structured_sparse_attention_b200 import inputs

pytestmark = pytest.mark.gpu


def ssa():
    import structured_sparse_attention_b200 as m
    return m


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def rows_of(cnt, row0, tok0=0):
    """(sequence, row) of the tokens tok0, tok0 + 1, ..."""
    return np.array([(b, r0 + i) for b, (c, r0) in enumerate(zip(cnt, row0)) for i in range(c)], np.int64).reshape(-1, 2)


def stored(cache, name):
    """Codes (unpacked) and scales, or the bf16 values, of a whole cache as numpy."""
    x = getattr(cache, name)
    if cache.format == "bf16":
        return f64(x), None
    return R.unpack(x.cpu().numpy(), cache.format), getattr(cache, name + "_scale").cpu().numpy()


def values(cache, name):
    c, e = stored(cache, name)
    return c if e is None else R.decode(c, e, cache.format)


def check_rounded(got, ref, size, fmt, scale=None):
    """got: values; ref: fp64 before the last rounding, off by up to 2^-19 size."""
    slack = 2.0 ** -19 * size
    if fmt == "bf16":
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * slack).all()
        return
    s = np.repeat(np.exp2(scale.astype(np.float64) - 127), R.GROUP, -1)
    z = (np.abs(ref) + slack) / s
    m, e = np.frexp(np.maximum(z, 1e-300))
    bits, low = (3, -9) if fmt == "e4m3" else (1, -1)
    half = np.exp2(np.maximum(e - 1 - bits, low).astype(np.float64)) / 2 * s
    assert (np.abs(got - ref) <= half + slack).all()
    top = np.abs(ref).reshape(*ref.shape[:-1], -1, R.GROUP).max(-1)
    big = size.reshape(top.shape + (R.GROUP,)).max(-1) * 2.0 ** -19
    s0 = np.exp2(scale.astype(np.float64) - 127)
    M = R.CODE_MAX[fmt]
    assert (top - big <= M * s0).all() and (top + big > M * s0 / 2).all()  # the smallest power of two


def run_append(fmt, d, Hq, Hkv, cnt, row0, S, *, norm=True, rotate=True, interleaved=False, pos=None, tok0=0, pad=0,
               joint=True, head_major=False, back=True, in_place=False, seed=0, big=1.0):
    m = ssa()
    n = tok0 + sum(cnt) + pad
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    new = lambda *s: (big * torch.randn(*s, device=dev(), generator=g)).bfloat16()
    if joint:
        x = new(n, Hq + 2 * Hkv, d)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:  # head-major, with room between the heads
        one = lambda h: new(h, n + 3, d)[:, :n].transpose(0, 1)
        q, k, v = one(Hq), one(Hkv), one(Hkv)
    src = [f64(a) for a in (q, k, v)]
    cache = m.KVCache(len(cnt), Hkv, S, d, fmt, device=dev())
    freqs = 10000.0 ** (-np.arange(d // 2) * 2.0 / d) if rotate else None
    w = [1 + 0.3 * np.random.default_rng(seed + i).standard_normal(d).astype(np.float32) for i in (1, 2)] if norm else [None] * 2
    T = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev())
    fill = lambda h: (torch.full((h, n, d), 7.0, device=dev(), dtype=torch.bfloat16).transpose(0, 1) if head_major
                      else torch.full((n, h, d), 7.0, device=dev(), dtype=torch.bfloat16))
    qo, ko, vo = (q, k, v) if in_place else (fill(Hq), fill(Hkv), fill(Hkv))
    ptr = t_i32(tok0 + np.concatenate([[0], np.cumsum(cnt)]))
    out = m.kv_append(cache, k, v, ptr, t_i32(row0), q=q, q_out=qo, pos=None if pos is None else t_i32(pos),
                      freqs=T(freqs), interleaved=interleaved, q_weight=T(w[0]), k_weight=T(w[1]), eps=1e-5,
                      k_out=ko if back else None, v_out=vo if back else None)
    at = rows_of(cnt, row0)
    live = slice(tok0, tok0 + len(at))
    P = at[:, 1] if pos is None else np.asarray(pos)[live]
    rq, sq = R.norm_rotate(src[0][live], P, w[0], 1e-5, freqs, interleaved)
    rk, sk = R.norm_rotate(src[1][live], P, w[1], 1e-5, freqs, interleaved)
    check_rounded(f64(out)[live], rq, sq, "bf16")
    ck, ek = stored(cache, "k")
    b, r = at[:, 0], at[:, 1]
    vk = values(cache, "k")[b, :, r]
    check_rounded(vk, rk, sk, fmt, None if ek is None else ek[b, :, r])
    cv, ev = stored(cache, "v")
    if fmt == "bf16":
        np.testing.assert_array_equal(cv[b, :, r], src[2][live])
    else:
        c, e = R.encode(src[2][live], fmt)
        np.testing.assert_array_equal(ev[b, :, r], e)
        np.testing.assert_array_equal(cv[b, :, r], c)
    if back:
        np.testing.assert_array_equal(f64(ko)[live], vk)
        np.testing.assert_array_equal(f64(vo)[live], values(cache, "v")[b, :, r])
    # nothing else is written: padding tokens and other rows
    if not in_place:
        for o in (out,) + ((ko, vo) if back else ()):
            rest = np.delete(f64(o), np.arange(tok0, tok0 + len(at)), 0)
            assert (rest == 7).all()
    for name in ("k", "v"):
        full = getattr(cache, name).clone()
        full[torch.from_numpy(b), :, torch.from_numpy(r)] = 0
        assert not full.any()
    # read back: exact, padding left alone
    k2, v2 = (torch.full((Hkv, n, d), 7.0, device=dev(), dtype=torch.bfloat16).transpose(0, 1) for _ in range(2))
    m.kv_read(cache, ptr, t_i32(row0), n, k_out=k2, v_out=v2)
    np.testing.assert_array_equal(f64(k2)[live], vk)
    np.testing.assert_array_equal(f64(v2)[live], values(cache, "v")[b, :, r])
    assert (np.delete(f64(k2), np.arange(tok0, tok0 + len(at)), 0) == 7).all()
    return cache


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_ragged(fmt, d, interleaved):
    run_append(fmt, d, 6, 2, [5, 0, 17, 1], [3, 0, 40, 63], 64, interleaved=interleaved, tok0=2, pad=5)


@pytest.mark.parametrize("fmt", R.FORMATS)
@pytest.mark.parametrize("n", [1, 2, 3, 5, 31, 33, 257, 4099])
def test_append_lengths(fmt, n):
    run_append(fmt, 128 if n % 2 else 64, 4, 1, [n], [1], n + 2, head_major=n > 100, joint=n < 100, seed=n)


@pytest.mark.parametrize("norm,rotate", [(False, True), (True, False), (False, False)])
def test_append_without_norm_or_rotation(norm, rotate):
    for fmt in R.FORMATS:
        run_append(fmt, 64, 3, 3, [9, 4], [0, 7], 20, norm=norm, rotate=rotate, back=False)


@pytest.mark.parametrize("fmt", R.FORMATS)
def test_append_positions_of_a_tree_and_in_place(fmt):
    pos = np.array([1000, 70000, 5, 104000, 0, 2000000000 // 16, 9], np.int32)
    run_append(fmt, 128, 5, 1, [4, 3], [10, 2], 30, pos=pos, in_place=True)


def test_append_many_heads_takes_several_rows_a_unit():
    # enough tokens that a unit takes 16 rows of one token
    run_append("e4m3", 64, 32, 8, [5000], [0], 5001, head_major=True, seed=3)
    run_append("e2m1", 128, 32, 8, [3001, 2777], [0, 100], 3100, seed=4)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_value_extremes(fmt):
    # zeros, tiny and huge groups, infinities and NaN, ties: V is stored without arithmetic
    m = ssa()
    g = np.random.default_rng(7)
    x = g.standard_normal((40, 1, 64)) * np.exp2(g.integers(-126, 110, (40, 1, 2))).repeat(32, 2)
    x[0] = 0
    x[1, 0, :32] = 448 * 2.0 ** 7
    x[2, 0, :32] = np.linspace(-6, 6, 32)
    x[3, 0, 5] = np.inf
    x[4, 0, 40] = np.nan
    x[5, 0, :32] = 3e38
    x[6, 0, 0], x[6, 0, 32:] = -0.0, 2.0 ** -133
    x[7, 0, :32] = np.arange(32) / 4.0
    x = R.bf16(x)
    t = torch.from_numpy(x).to(dev()).bfloat16()
    cache = m.KVCache(1, 1, 40, 64, fmt, device=dev())
    ko, vo = torch.empty_like(t), torch.empty_like(t)
    m.kv_append(cache, torch.zeros_like(t), t, t_i32([0, 40]), t_i32([0]), k_out=ko, v_out=vo)
    c, e = R.encode(x, fmt)
    cv, ev = stored(cache, "v")
    np.testing.assert_array_equal(ev[0, 0], e[:, 0])
    np.testing.assert_array_equal(cv[0, 0], c[:, 0])
    want = R.decode(c, e, fmt)
    np.testing.assert_array_equal(f64(vo), want)
    k2, v2 = m.kv_read(cache, t_i32([0, 40]), t_i32([0]), 40)
    np.testing.assert_array_equal(f64(v2), want)
    assert not k2.any()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_every_code_at_every_scale_reads_back_exactly(fmt):
    m = ssa()
    hi = {"e4m3": 134, "e2m1": 140}[fmt]
    scales = np.array(list(range(16, hi + 1)), np.uint8)
    codes = np.array([c for c in range(256 if fmt == "e4m3" else 16) if fmt == "e2m1" or (c & 127) != 127], np.uint8)
    codes = np.resize(codes, 256)  # 4 rows of 64 cover every code
    rows = np.tile(codes.reshape(4, 64), (len(scales), 1))
    e = np.repeat(scales, 4)[:, None].repeat(2, 1)
    n = len(rows)
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a)[None, None]).to(dev())
    cache = m.KVCache.from_tensors(T(R.pack(rows, fmt)), T(R.pack(rows, fmt)), T(e), T(e), format=fmt)
    k, v = m.kv_read(cache, t_i32([0, n]), t_i32([0]), n)
    want = R.decode(rows, e, fmt)
    np.testing.assert_array_equal(f64(k)[:, 0], want)
    np.testing.assert_array_equal(f64(v)[:, 0], want)


def test_bad_descriptors_are_reported_and_skipped():
    m = ssa()
    d, S = 64, 16
    k = torch.ones(8, 1, d, device=dev(), dtype=torch.bfloat16)
    for ptr, row0, pos in [([0, 4, 3], [0, 0], None), ([0, 4, 9], [0, 0], None), ([0, 4, 8], [0, 13], None),
                           ([0, 4, 8], [-1, 0], None), ([-2, 4, 8], [0, 0], None), ([0, 4, 8], [2147483647, 0], None),
                           ([0, 4, 8], [0, 0], [0, 1, 2, 3, 4, -5, 6, 7])]:
        cache = m.KVCache(2, 1, S, d, "bf16", device=dev())
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        m.kv_append(cache, k, k, t_i32(ptr), t_i32(row0), pos=None if pos is None else t_i32(pos), status=status, check=False)
        torch.cuda.synchronize()
        assert int(status) == -1, (ptr, row0)
        assert set(cache.k.unique().tolist()) <= {0.0, 1.0}
        if pos is None:
            out = torch.zeros(8, 1, d, device=dev(), dtype=torch.bfloat16)
            with pytest.raises(m.SSAError):
                m.kv_read(cache, t_i32(ptr), t_i32(row0), 8, k_out=out, v_out=torch.zeros_like(out))
    # a skipped position leaves its neighbours written
    assert cache.k[1, 0, 0, 0] == 1 and cache.k[1, 0, 1, 0] == 0 and cache.k[1, 0, 2, 0] == 1


def test_no_tokens_is_a_no_op():
    m = ssa()
    cache = m.KVCache(1, 1, 4, 64, "e4m3", device=dev())
    e = torch.empty(0, 1, 64, device=dev(), dtype=torch.bfloat16)
    m.kv_append(cache, e, e, t_i32([0, 0]), t_i32([0]))
    k, v = m.kv_read(cache, t_i32([0, 0]), t_i32([0]), 0)
    assert k.shape == (0, 1, 64) and not cache.k.any()


def test_rows_past_32_bits():
    # the last rows of a cache of more than 2^31 elements
    m = ssa()
    B, H, S, d = 2, 16, 600000, 128
    cache = m.KVCache(B, H, S, d, "bf16", device=dev())
    assert cache.k.numel() > 2 ** 31
    x = torch.randn(6, H, d, device=dev()).bfloat16()
    m.kv_append(cache, x, 2 * x, t_i32([0, 3, 6]), t_i32([1, S - 3]))
    assert torch.equal(cache.k[1, :, S - 3:], x[3:].transpose(0, 1))
    assert torch.equal(cache.v[0, :, 1:4], 2 * x[:3].transpose(0, 1))
    k, v = m.kv_read(cache, t_i32([0, 3, 6]), t_i32([1, S - 3]), 6)
    assert torch.equal(k, x) and torch.equal(v, 2 * x)


def test_captured_replayed_and_on_another_stream():
    m = ssa()
    d, H, S, n = 128, 2, 64, 9
    cache = m.KVCache(1, H, S, d, "e4m3", device=dev())
    x = torch.randn(n, 3 * H, d, device=dev()).bfloat16()
    q, k, v = x[:, :H], x[:, H:2 * H], x[:, 2 * H:]
    qo, ko, vo = (torch.zeros(n, H, d, device=dev(), dtype=torch.bfloat16) for _ in range(3))
    freqs = torch.from_numpy(10000.0 ** (-np.arange(d // 2) * 2.0 / d)).to(dev())
    ptr, row0 = t_i32([0, n]), t_i32([0])
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    kw = dict(q=q, q_out=qo, freqs=freqs, k_out=ko, v_out=vo, status=status, check=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.kv_append(cache, k, v, ptr, row0, stream=side, **kw)
    side.synchronize()
    want = [t.clone() for t in (qo, ko, vo, cache.k, cache.v_scale)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.kv_append(cache, k, v, ptr, row0, **kw)
    for t in (qo, ko, vo, cache.k, cache.v_scale):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (qo, ko, vo, cache.k, cache.v_scale)):
        assert torch.equal(a, b)
    row0.fill_(20)  # the descriptors are read at replay
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.v[0, :, 20:29], cache.v[0, :, 0:9])
    assert int(status) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt,top", [("e4m3", 134), ("e2m1", 140)])
def test_scale_bytes_out_of_range_are_reported(fmt, top, d):
    m = ssa()
    B, S = 2, 50
    cache = m.KVCache(B, 3, S, d, fmt, device=dev())
    ptr, row0 = t_i32([0, 30, 50]), t_i32([4, 7])
    for t in (cache.k_scale, cache.v_scale):
        for E in (0, 1, 16, 113, top, 255):
            t[1, 2, 20, -1] = E
            m.kv_read(cache, ptr, row0, 50)
        for E in (top + 1, 142, 254):
            t[1, 2, 20, -1] = E
            with pytest.raises(m.SSAError) as e:
                m.kv_read(cache, ptr, row0, 50)
            assert e.value.code == -1
        t[1, 2, 20, -1] = 127
        t[1, 2, 40, -1] = top + 1  # a row that the call does not read
        m.kv_read(cache, ptr, row0, 50)
