"""The 4-bit K/V cache on the GPU against the float64 oracle.

Quantisation and reading back are exact: codes stand for equal values, scales are equal bytes.

Attention, per element, with A = sum_j p_j |v_j| (the oracle's spread), n visible positions and
D = head_dim:
  |out - ref| <= 2^-8 |ref|            the bf16 output, rounded once
               + (2^-11 + 2 dz + n 2^-22) A + 2^-32 sum_j |v_j| + 2^-133
where a probability is rounded to f16 (2^-11; held as P = 2^(7 + x - m) at a running maximum m
that some position has set, so l >= 2^7, while P below 2^-14 lies on f16's grid of 2^-24, half a
step of which is 2^-25, and 2^-25 / 2^7 = 2^-32 for each position: rescaling and joining only
multiply both by factors <= 1), dz bounds a score's error: D products summed in
f32, each partial sum off by at most 2^-23 of sum |q k| (the queries' power of two and the
cached values are exact), and n 2^-22 covers the f32 sums over the positions of the numerator
and the denominator, ex2.approx (2^-22) and the joins. The log-sum-exp is off by at most
  dz + n 2^-23 + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import kv4 as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    from block_kv_cache_b200 import fdllm
    c = fdllm.Context(0)
    yield c
    c.close()


def fdl():
    from block_kv_cache_b200 import fdllm
    return fdllm


def host(cache):
    return [t.cpu().numpy() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]


def random_cache(b, hkv, L, d, seed, fill=None):
    """A cache of rows with a few large key channels, quantised by the oracle; `fill` bytes
    everywhere instead."""
    rng = np.random.default_rng(seed)
    parts = []
    for key in (True, False):
        x = rng.standard_normal((b, hkv, L, d))
        if key:
            x *= np.where(rng.random(d) > 0.94, 6.0, 0.7)
        parts += list(O.kv4_quantise(x))
    if fill is not None:
        for p in parts:
            p[...] = fill
    return fdl().Kv4Cache(*(torch.from_numpy(p).cuda() for p in parts))


# ------------------------------------------------------------------------ quantisation
def store_rows(ctx, x, dtype):
    """(codes, scales) after storing rows x [n, d] as both K and V of one head."""
    t = torch.from_numpy(x).to(dtype).cuda()[None, :, None, :].contiguous()
    c = fdl().Kv4Cache.empty(1, 1, x.shape[0], x.shape[1])
    ctx.kv4_store(t, t, c, 0)
    k, ks, v, vs = host(c)
    np.testing.assert_array_equal(k, v)
    np.testing.assert_array_equal(ks, vs)
    return k[0, 0], ks[0, 0]


def check_quantised(got, x):
    codes, scales = O.kv4_quantise(x)
    np.testing.assert_array_equal(got[1], scales)
    np.testing.assert_array_equal(O.kv4_values(*got), O.kv4_values(codes, scales))


def test_every_bf16_value_under_every_scale(ctx):
    """All bf16 magnitudes (both signs) below the largest of their group, for a largest value
    that gives each of the 126 scales."""
    every = (np.arange(0x0000, 0x7f80, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)
    for s in range(1, 127):
        top = 6 * K.E4M3[s]
        lo, hi = 2.0 ** -6 * K.E4M3[s], top
        x = every[(every >= lo) & (every <= hi)]
        x = np.concatenate([x, -x])
        x = np.concatenate([x, np.zeros(-len(x) % 15)]).reshape(-1, 15)
        g = np.concatenate([np.full((len(x), 1), top), x], 1)
        g = np.concatenate([g, np.zeros((-len(g) % 8, 16))]).reshape(-1, 128)
        check_quantised(store_rows(ctx, g, torch.bfloat16), g)


def test_f32_values_next_to_the_borders(ctx):
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    groups = []
    for s in range(1, 127):
        b = (borders * np.float32(K.E4M3[s])).astype(np.float32)          # exact
        x = np.concatenate([np.nextafter(b, np.float32(0)), b,
                            np.nextafter(b, np.float32(1e9))]).astype(np.float64)
        x = np.concatenate([x, -x, np.zeros(3)]).reshape(3, 15)
        groups.append(np.concatenate([np.full((3, 1), 6 * K.E4M3[s]), x], 1))
        # largest values next to the borders of two scales
        if s < 126:
            mid = np.float32(3 * (K.E4M3[s] + K.E4M3[s + 1]))
            for m in (np.nextafter(mid, np.float32(0)), mid, np.nextafter(mid, np.float32(1e9))):
                groups.append(np.concatenate([[[m]], np.full((1, 15), m / 3)], 1))
    g = np.concatenate(groups).astype(np.float32).astype(np.float64)
    g = np.concatenate([g, np.zeros((-len(g) % 4, 16))]).reshape(-1, 64)
    check_quantised(store_rows(ctx, g, torch.float32), g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinities_nan_and_tiny_groups(ctx, dtype):
    x = np.zeros((8, 128))
    x[0, 3], x[0, 5], x[0, 6] = np.inf, -np.inf, 5.0
    x[1, 17] = np.nan
    x[1, 18] = np.inf
    x[2] = 2.0 ** -12
    x[3] = -2.0 ** -130
    x[4, :16] = 3e38
    x[4, 16:32] = -3e38
    x[5, :16] = 2688.0
    x[6] = 3 * 2.0 ** -9
    x = torch.from_numpy(x).to(dtype).double().numpy()
    got = store_rows(ctx, x, dtype)
    check_quantised(got, x)
    v = O.kv4_values(*got)
    assert np.isnan(v[1, 16:32]).all() and np.isfinite(np.delete(v[1], range(16, 32))).all()


# ---------------------------------------------------------------- placement and strides
def fresh(b, n, hkv, d, dtype, layout, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "token":
        return torch.randn((b, n, hkv, d), generator=g, device="cuda").to(dtype)
    if layout == "head":                                    # a slice of a head-major buffer
        x = torch.randn((b, hkv, n + 5, d), generator=g, device="cuda").to(dtype)
        return x[:, :, 2:2 + n].transpose(1, 2)
    if layout == "sliced":                                  # part of a wider row, as of q|k|v
        x = torch.randn((b, n, hkv + 3, d), generator=g, device="cuda").to(dtype)
        return x[:, :, 1:1 + hkv]
    x = torch.randn((1, n, hkv, d), generator=g, device="cuda").to(dtype)
    return x.expand(b, n, hkv, d)                           # "shared": one prompt for all


@pytest.mark.parametrize("b,hkv,d,L,start,n", [
    (1, 32, 128, 768, 512, 32), (2, 4, 128, 300, 17, 211), (3, 2, 64, 131, 130, 1),
    (1, 1, 64, 1, 0, 1), (2, 3, 128, 40, 0, 40), (5, 7, 64, 67, 3, 61), (1, 1, 128, 4097, 5, 4090),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["token", "head", "sliced", "shared"])
def test_store_and_read_back(ctx, b, hkv, d, L, start, n, dtype, layout):
    if layout == "shared" and b == 1:
        pytest.skip("nothing to share")
    c = random_cache(b, hkv, L, d, seed=1, fill=0x5a)
    before = host(c)
    k, v = fresh(b, n, hkv, d, dtype, layout, 2), fresh(b, n, hkv, d, dtype, layout, 3)
    ctx.kv4_store(k, v, c, start)
    after = host(c)
    want = []
    for x, codes, scales in ((k, 0, 1), (v, 2, 3)):
        q = O.kv4_quantise(x.double().cpu().numpy().transpose(0, 2, 1, 3))
        np.testing.assert_array_equal(after[scales][:, :, start:start + n], q[1])
        vals = O.kv4_values(*q)
        np.testing.assert_array_equal(
            O.kv4_values(after[codes][:, :, start:start + n],
                         after[scales][:, :, start:start + n]), vals)
        want.append(vals.transpose(0, 2, 1, 3))
        for i in (codes, scales):                            # nothing else is written
            np.testing.assert_array_equal(np.delete(after[i], range(start, start + n), 2),
                                          np.delete(before[i], range(start, start + n), 2))
    # read back in both types, and into a head-major buffer with its surroundings kept
    for dt in (torch.bfloat16, torch.float32):
        for got, w in zip(ctx.kv4_load(c, start, n, dtype=dt), want):
            assert got.dtype == dt and got.shape == (b, n, hkv, d)
            np.testing.assert_array_equal(got.double().cpu().numpy(), w)
        buf = torch.full((b, hkv, n + 3, d), 7.0, dtype=dt, device="cuda")
        ctx.kv4_load(c, start, n, v_out=buf[:, :, 1:1 + n].transpose(1, 2))
        g = buf.double().cpu().numpy()
        np.testing.assert_array_equal(g[:, :, 1:1 + n].transpose(0, 2, 1, 3), want[1])
        assert (g[:, :, 0] == 7).all() and (g[:, :, n + 1:] == 7).all()


def test_load_reads_nan_scales_and_whole_cache(ctx):
    c = random_cache(1, 2, 9, 64, seed=4)
    c.v_scale[0, 1, 3, 2] = 127
    k, v = ctx.kv4_load(c)
    kc, ks, vc, vs = host(c)
    np.testing.assert_array_equal(v.double().cpu().numpy(),
                                  O.kv4_values(vc, vs).transpose(0, 2, 1, 3))
    assert torch.isnan(v[0, 3, 1, 32:48]).all() and not torch.isnan(k).any()
    np.testing.assert_array_equal(k.double().cpu().numpy(),
                                  O.kv4_values(kc, ks).transpose(0, 2, 1, 3))


# --------------------------------------------------------------------------- attention
def check_attention(q, cache, out, lse, start, kv_len=None, window=(-1, -1), sinks=0, scale=None,
                    seqs=None):
    b, B, hq, d = q.shape
    kc, ks, vc, vs = host(cache)
    qn, on, ln = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    sc = d ** -0.5 if scale is None else scale
    for i in seqs if seqs is not None else range(b):
        seen = O.kv4_visible(cache.seq_len, start, B, None if kv_len is None else kv_len[i],
                             window, sinks)
        n = int(seen.sum())
        k, v = O.kv4_values(kc[i][:, seen], ks[i][:, seen]), O.kv4_values(vc[i][:, seen],
                                                                         vs[i][:, seen])
        ref, rl, spread = O.kv4_attention(qn[i], k, v, np.ones(n, bool), sc)
        if n == 0:
            assert (on[i] == 0).all() and np.isneginf(ln[i]).all()
            continue
        # a bound of sum |q k| over the head dims, by Cauchy
        dz = d * 2.0 ** -23 * sc * np.linalg.norm(qn[i], axis=-1).max() * \
            np.linalg.norm(k, axis=-1).max()
        grid = np.repeat(np.abs(v).sum(1), hq // cache.n_kv_heads, 0) * 2.0 ** -32 + 2.0 ** -133
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * dz + n * 2.0 ** -22) * spread + grid
        bad = np.abs(on[i] - ref) - tol
        assert bad.max() <= 0, (i, bad.max(), np.abs(on[i] - ref).max())
        ltol = dz + n * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(rl))
        assert (np.abs(ln[i] - rl) <= ltol).all(), (i, np.abs(ln[i] - rl).max())


def queries(b, B, hq, d, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((b, B, hq, d), generator=g, device="cuda") * size).to(torch.bfloat16)


SHAPES = [  # b, Hq, Hkv, d, L, start, B
    (1, 4, 4, 128, 128, 64, 32),
    (1, 32, 32, 128, 768, 512, 32),
    (2, 28, 4, 128, 1024, 512, 32),      # 224 packed rows
    (3, 8, 2, 64, 53, 37, 5),
    (1, 2, 2, 128, 1, 0, 1),
    (1, 3, 3, 64, 129, 0, 128),
    (2, 4, 4, 128, 1020, 1000, 17),
    (1, 7, 1, 128, 5000, 4999, 1),       # a single token, several splits
    (2, 16, 1, 64, 777, 3, 1),
    (1, 40, 8, 128, 95, 31, 33),         # 165 packed rows, odd group
    (4, 6, 6, 64, 31, 0, 31),
    (1, 1, 1, 128, 33, 32, 1),
    (70, 2, 2, 64, 40, 8, 8),
    (1, 8, 8, 128, 2048, 1024, 128),
    (2, 32, 8, 128, 2300, 1000, 32),     # 16 units of 128 rows: clusters of 2, joined twice
    (2, 16, 8, 64, 2300, 1000, 64),
    (5, 16, 4, 128, 2000, 77, 32),       # 20 units of 128 rows: larger clusters
    (6, 31, 1, 128, 3001, 2990, 11),     # 341 rows: two chunks, the last of 170
    (6, 32, 4, 64, 701, 64, 32),         # 24 units of 256 rows
    (6, 30, 2, 128, 901, 800, 17),  # 255 rows
]


@pytest.mark.parametrize("b,hq,hkv,d,L,start,B", SHAPES)
def test_attention_shapes(ctx, b, hq, hkv, d, L, start, B):
    c, q = random_cache(b, hkv, L, d, seed=11), queries(b, B, hq, d, 12)
    out, lse = ctx.kv4_attention(q, c, start, want_lse=True)
    check_attention(q, c, out, lse, start, seqs=range(min(b, 3)))
    ctx.device_status()
    # the same bits again, and without the log-sum-exp
    assert torch.equal(ctx.kv4_attention(q, c, start), out)


@pytest.mark.parametrize("b,hq,hkv,d,L,start,B", [
    (5, 8, 2, 128, 700, 300, 16), (5, 4, 4, 64, 260, 100, 32), (5, 7, 1, 128, 3000, 2999, 1),
    (5, 28, 4, 128, 400, 200, 32)])
def test_attention_kv_len(ctx, b, hq, hkv, d, L, start, B):
    """Lengths of none, one, part of a step, all, and beyond either end (clamped)."""
    lens = [0, 1, L // 2 + 3, L + 1000, -7]
    c, q = random_cache(b, hkv, L, d, seed=21), queries(b, B, hq, d, 22)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = ctx.kv4_attention(q, c, start, kv_len=n, want_lse=True)
    check_attention(q, c, out, lse, start, kv_len=[max(0, min(L, x)) for x in lens])


WINDOWS = [((100, 50), 4), ((0, 0), 0), ((0, 0), 1), ((5, -1), 3), ((-1, 7), 9), ((40, 3), 500),
           ((2147483647, 0), 0), ((33, 31), 32), ((10, 10), 2147483647)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("hq,hkv,d,L,start,B", [
    (4, 4, 128, 600, 290, 32), (8, 2, 64, 333, 200, 7), (14, 2, 128, 500, 499, 1),
    (28, 4, 128, 640, 320, 32), (4, 4, 128, 200, 0, 16)])
def test_attention_window_and_sinks(ctx, hq, hkv, d, L, start, B, window, sinks):
    lens = [L, start + B // 2, 1, start + B + 1]
    c, q = random_cache(4, hkv, L, d, seed=31), queries(4, B, hq, d, 32)
    out, lse = ctx.kv4_attention(q, c, start, window=window, sinks=sinks, want_lse=True,
                                 kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check_attention(q, c, out, lse, start, lens, window, sinks)


def test_attention_sees_nothing(ctx):
    """A window behind the sequence's length, and no sinks: zeros, -inf."""
    c, q = random_cache(2, 2, 300, 64, seed=41), queries(2, 8, 4, 64, 42)
    n = torch.tensor([50, 0], dtype=torch.int32, device="cuda")
    out, lse = ctx.kv4_attention(q, c, 200, kv_len=n, window=(10, 10), want_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("hq,hkv,d,L,start,B", [
    (4, 4, 128, 600, 290, 32), (7, 1, 128, 4000, 2000, 1), (28, 4, 128, 640, 320, 32),
    (8, 2, 64, 333, 200, 7)])
def test_what_is_not_seen_may_hold_anything(ctx, hq, hkv, d, L, start, B):
    """NaN scales and large codes outside the visible positions change no bit."""
    c, q = random_cache(2, hkv, L, d, seed=51), queries(2, B, hq, d, 52)
    lens, window, sinks = [L - 37, start + 5], (50, 21), 3
    kw = dict(kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"), window=window,
              sinks=sinks, want_lse=True)
    clean = ctx.kv4_attention(q, c, start, **kw)
    for i in range(2):
        unseen = torch.from_numpy(~O.kv4_visible(L, start, B, lens[i], window, sinks)).cuda()
        for t in (c.k, c.k_scale, c.v, c.v_scale):
            t[i][:, unseen] = 0x7f if t.shape[-1] == d // 16 else 0xff
    dirty = ctx.kv4_attention(q, c, start, **kw)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    check_attention(q, c, *dirty, start, lens, window, sinks)


def test_nan_reaches_only_what_sees_it(ctx):
    c, q = random_cache(2, 2, 100, 128, seed=61), queries(2, 16, 4, 128, 62)
    c.k_scale[1, 0, 40, 3] = 127            # a key of sequence 1, kv head 0
    c.v_scale[1, 1, 41, 2] = 127            # a value of kv head 1: dims 32..47
    out, lse = ctx.kv4_attention(q, c, 32, want_lse=True)
    assert not torch.isnan(out[0]).any() and not torch.isnan(lse[0]).any()
    assert torch.isnan(out[1, :, :2]).all() and torch.isnan(lse[1, :2]).all()
    assert torch.isnan(out[1, :, 2:, 32:48]).all() and not torch.isnan(lse[1, 2:]).any()
    assert not torch.isnan(out[1, :, 2:, :32]).any() and not torch.isnan(out[1, :, 2:, 48:]).any()


@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -40, 1e-3, 30.0])
@pytest.mark.parametrize("hq,L", [(4, 300), (28, 300)])
def test_attention_query_sizes(ctx, size, hq, L):
    """Queries far below and above 1: uniform to nearly one-hot probabilities."""
    c, q = random_cache(1, 4, L, 128, seed=71), queries(1, 32, hq, 128, 72, size)
    out, lse = ctx.kv4_attention(q, c, 100, want_lse=True)
    check_attention(q, c, out, lse, 100)


def test_attention_query_rows_of_mixed_sizes(ctx):
    """Rows, and elements within a row, many powers of two apart."""
    q = queries(1, 32, 4, 128, 73)
    q = (q.float() * torch.exp2((torch.arange(32, device="cuda") % 13 - 9.0))[None, :, None, None]
         * torch.exp2(-(torch.arange(128, device="cuda") % 20.0))).to(torch.bfloat16)
    q[0, 3] = 0
    c = random_cache(1, 4, 200, 128, seed=74)
    out, lse = ctx.kv4_attention(q, c, 100, want_lse=True)
    check_attention(q, c, out, lse, 100)


@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_attention_scale(ctx, scale):
    c, q = random_cache(1, 2, 200, 64, seed=75), queries(1, 9, 4, 64, 76)
    out, lse = ctx.kv4_attention(q, c, 100, want_lse=True, scale=scale)
    check_attention(q, c, out, lse, 100, scale=float(np.float32(scale)))


def test_scores_that_grow_along_the_sequence(ctx):
    """The running maximum is raised again and again."""
    L, d = 700, 128
    rng = np.random.default_rng(81)
    u = rng.standard_normal(d)
    k = np.outer(np.linspace(-20, 20, L), u)[None, None] + rng.standard_normal((1, 2, L, d))
    v = rng.standard_normal((1, 2, L, d))
    c = fdl().Kv4Cache(*(torch.from_numpy(p).cuda()
                         for p in (*O.kv4_quantise(k), *O.kv4_quantise(v))))
    q = torch.from_numpy(u / 4 + rng.standard_normal((1, 20, 4, d)) / 4).to(torch.bfloat16).cuda()
    out, lse = ctx.kv4_attention(q, c, 300, want_lse=True)
    check_attention(q, c, out, lse, 300)


def test_positions_behind_32_bits(ctx):
    """Byte offsets above 2^32 in the codes: 72 million positions of one head."""
    L, d, hkv = 72_000_000, 128, 1
    codes = torch.zeros((1, hkv, L, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, hkv, L, d // 16), dtype=torch.uint8, device="cuda")
    c = fdl().Kv4Cache(codes, scales, codes.clone(), scales.clone())
    n, start = 300, L - 310
    k, v = fresh(1, n, hkv, d, torch.bfloat16, "token", 91), fresh(1, n, hkv, d, torch.bfloat16,
                                                                   "token", 92)
    ctx.kv4_store(k, v, c, start)
    want = [O.kv4_quantise(x.double().cpu().numpy().transpose(0, 2, 1, 3)) for x in (k, v)]
    got = ctx.kv4_load(c, start, n)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.double().cpu().numpy(),
                                      O.kv4_values(*w).transpose(0, 2, 1, 3))
    assert not c.k[:, :, :1000].any() and not c.k[:, :, start - 1000:start].any()
    q = queries(1, 4, 2, d, 93)
    out, lse = ctx.kv4_attention(q, c, L - 100, window=(150, -1), sinks=5, want_lse=True)
    # the same few positions in a small cache
    sub = fdl().Kv4Cache(*(torch.cat([t[:, :, :5], t[:, :, L - 250:]], 2).contiguous()
                           for t in (c.k, c.k_scale, c.v, c.v_scale)))
    check_attention(q, sub, out, lse, 5)


# ------------------------------------------------------- streams, graphs, workspaces
def test_other_stream_and_given_buffers(ctx):
    c, q = random_cache(1, 4, 3000, 128, seed=101), queries(1, 1, 28, 128, 102)
    want, wl = ctx.kv4_attention(q, c, 2999, want_lse=True)
    need = ctx.kv4_attention_workspace_bytes(ctx.kv4_attn_desc(q, c, 2999))
    assert need > 16                                         # several splits
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.full_like(want, 9), torch.full_like(wl, 9)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    ctx.kv4_attention(q, c, 2999, out=out, lse=lse, ws=ws, stream=s)
    again = ctx.kv4_attention(q, c, 2999, stream=s)
    k, v = fresh(1, 5, 4, 128, torch.bfloat16, "token", 103), fresh(1, 5, 4, 128, torch.bfloat16,
                                                                    "token", 104)
    s.wait_stream(torch.cuda.current_stream())
    ctx.kv4_store(k, v, c, 10, stream=s)
    back = ctx.kv4_load(c, 10, 5, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(again, want)
    np.testing.assert_array_equal(
        back[0].double().cpu().numpy(),
        O.kv4_values(*O.kv4_quantise(k.double().cpu().numpy())))
    with pytest.raises(fdl().FdlError) as e:
        ctx.kv4_attention(q, c, 2999, ws=ws[:need - 16])
    assert e.value.code == fdl().FDL_EWORKSPACE


def test_two_calls_at_once(ctx):
    """Calls on two streams, each with its own scratch, do not disturb one another."""
    cs = [random_cache(1, 2, 4096, 128, seed=111 + i) for i in range(2)]
    qs = [queries(1, 8, 8, 128, 113 + i) for i in range(2)]
    want = [ctx.kv4_attention(qs[i], cs[i], 2048) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(ctx.kv4_attention(qs[i], cs[i], 2048, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_captured_step_replays_on_new_inputs(ctx):
    """Store, attention and read-back captured once; two graphs, replayed in turn with other
    rows, queries and lengths."""
    b, hkv, hq, d, L, start, B = 2, 2, 8, 128, 900, 512, 32
    graphs, state = [], []
    for i in range(2):
        c, q = random_cache(b, hkv, L, d, seed=121 + i), queries(b, B, hq, d, 123 + i)
        k, v = (fresh(b, B, hkv, d, torch.bfloat16, "token", s + i) for s in (125, 127))
        n = torch.tensor([L, 600], dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ctx.kv4_store(k, v, c, start)
            ctx.kv4_attention(q, c, start, kv_len=n)
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(g):
            ctx.kv4_store(k, v, c, start)
            out, lse = ctx.kv4_attention(q, c, start, kv_len=n, want_lse=True)
            back = ctx.kv4_load(c, start, B)
        graphs.append(g)
        state.append((c, q, k, v, n, out, lse, back))
    for r in range(2):
        for i in (1, 0):
            c, q, k, v, n, out, lse, back = state[i]
            q.copy_(queries(b, B, hq, d, 200 + r))
            k.copy_(fresh(b, B, hkv, d, torch.bfloat16, "token", 300 + r))
            n.copy_(torch.tensor([0 if r else 37, L - r], dtype=torch.int32))
            graphs[i].replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(
                back[0].double().cpu().numpy(),
                O.kv4_values(*O.kv4_quantise(k.double().cpu().numpy())))
            check_attention(q, c, out, lse, start, n.tolist())


# -------------------------------------------------------------- used together
def test_a_cached_step_against_the_bf16_path(ctx):
    """A refresh's rows and then a block's rows stored in 4 bits; the attention over the cache
    equals the bf16 attention over the values read back, within both kernels' rounding."""
    b, hq, hkv, d, L, start, B = 2, 8, 2, 128, 640, 320, 32
    c = fdl().Kv4Cache.empty(b, hkv, L, d)
    for s, n, seed in ((0, L, 131), (start, B, 133)):
        ctx.kv4_store(fresh(b, n, hkv, d, torch.bfloat16, "head", seed),
                      fresh(b, n, hkv, d, torch.bfloat16, "head", seed + 1), c, s)
    q = queries(b, B, hq, d, 135)
    out, lse = ctx.kv4_attention(q, c, start, want_lse=True)
    check_attention(q, c, out, lse, start)
    kc, vc = (torch.empty((b, hkv, L, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx.kv4_load(c, k_out=kc.transpose(1, 2), v_out=vc.transpose(1, 2))
    ref, rl = ctx.dualcache_attention(q, kc, vc, start, want_lse=True)
    torch.cuda.synchronize()
    # outputs of at most ~1, each rounded to bf16 once, bf16 probabilities on one side
    assert (out.float() - ref.float()).abs().max() <= 2 * 2.0 ** -8 + 2.0 ** -7
    assert (lse - rl).abs().max() <= 2e-3


def test_binding_refusals(ctx):
    F = fdl()
    c, q = random_cache(2, 2, 64, 128, seed=141), queries(2, 8, 4, 128, 142)
    k = fresh(2, 8, 2, 128, torch.bfloat16, "token", 143)
    with pytest.raises(ValueError):
        ctx.kv4_store(k[:1], k[:1], c, 0)                    # another batch
    with pytest.raises(ValueError):
        ctx.kv4_store(k, k.transpose(0, 1).contiguous().transpose(0, 1), c, 0)   # other strides
    with pytest.raises(ValueError):
        ctx.kv4_store(k, None, c, 0)
    with pytest.raises(ValueError):
        ctx.kv4_store(k[..., :64], k[..., :64], c, 0)
    with pytest.raises(TypeError):
        ctx.kv4_store(k, k.float(), c, 0)
    with pytest.raises(TypeError):
        ctx.kv4_store(k.half(), k.half(), c, 0)
    with pytest.raises(ValueError):
        ctx.kv4_store(k[..., ::2], k[..., ::2], c, 0)        # head_dim not contiguous
    with pytest.raises(F.FdlError):
        ctx.kv4_store(k, k, c, 57)                           # past the end
    with pytest.raises(F.FdlError):
        ctx.kv4_load(c, 60, 5)
    with pytest.raises(ValueError):
        ctx.kv4_load(c, 64)
    with pytest.raises(TypeError):
        ctx.kv4_attention(q.float(), c, 0)
    with pytest.raises(ValueError):
        ctx.kv4_attention(q[:1], c, 0)
    with pytest.raises(ValueError):
        ctx.kv4_attention(q, c, 0, kv_len=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        ctx.kv4_attention(q, c, 0, kv_len=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ctx.kv4_attention(q.transpose(1, 2).contiguous().transpose(1, 2), c, 0)
    with pytest.raises(ValueError):
        ctx.kv4_attention(q, c, 0, out=q.new_empty((2, 8, 4, 64)))
    with pytest.raises(F.FdlError):
        ctx.kv4_attention(q, c, 57)
    with pytest.raises(F.FdlError):
        ctx.kv4_attention(q, c, 0, out=q)
    with pytest.raises(ValueError):
        F.Kv4Cache(c.k, c.k_scale, c.v, c.v_scale[..., :4].contiguous())
    with pytest.raises(ValueError):
        ctx.kv4_store(k, k, c, 1 << 32)                      # not position 0
    with pytest.raises(ValueError):
        ctx.kv4_load(c, 1 << 32, 5)


@pytest.mark.parametrize("b,hq,hkv", [(24, 28, 4), (8, 32, 8)])   # alone, clusters of 2
def test_a_wait_that_runs_out_is_reported(b, hq, hkv):
    """Many query rows, waits limited to 1 ns: the kernel ends, and either no wait ran out (a
    poll may last until its barrier is there) and the result is right, or the host reads
    FDL_ETIMEOUT; a new context computes the same call."""
    F = fdl()
    c, q = random_cache(b, hkv, 500, 128, seed=151), queries(b, 32, hq, 128, 152)
    x = F.Context(0)
    x.set_wait_timeout(1)
    out, lse = x.kv4_attention(q, c, 200, want_lse=True)
    try:
        x.device_status()
    except F.FdlError as e:
        assert e.code == F.FDL_ETIMEOUT
    else:
        check_attention(q, c, out, lse, 200, seqs=range(2))
    x.close()
    torch.cuda.synchronize()
    x = F.Context(0)
    out, lse = x.kv4_attention(q, c, 200, want_lse=True)
    check_attention(q, c, out, lse, 200, seqs=range(2))
    x.device_status()
    x.close()


# ------------------------------------------------------- scores of any finite size
EXACT_SHAPES = [  # b, Hq, Hkv, d, L, start, B
    (1, 4, 4, 128, 300, 100, 32),        # few rows, joined over a cluster
    (2, 6, 3, 64, 333, 0, 9),
    (1, 7, 1, 128, 5000, 4999, 1),       # ... and in the workspace
    (24, 28, 4, 128, 200, 100, 32),      # many rows: two tiles, one block
    (8, 32, 8, 128, 500, 200, 32),       # one tile, a cluster of 2
    (38, 32, 8, 64, 90, 20, 32),         # one tile, one block
    (2, 32, 8, 128, 2300, 1000, 32),     # ... and in the workspace
]


def exact_scores(b, hq, hkv, d, L, B, seed, power):
    """Keys that are multiples of 0.5 up to 6 and queries that are whole numbers up to 8 times
    2^power: every partial sum of a score is a multiple of half that power below 2^14 of it, so
    f32 holds it whatever the order."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (2, b, hkv, L, d // 2), dtype=np.uint8)
    scales = np.full((2, b, hkv, L, d // 16), 0x38, np.uint8)               # 1.0
    c = fdl().Kv4Cache(*(torch.from_numpy(x).cuda()
                         for x in (codes[0], scales[0], codes[1], scales[1])))
    q = torch.from_numpy(rng.integers(-8, 9, (b, B, hq, d)) * 2.0 ** power).to(torch.bfloat16).cuda()
    return c, q


def check_exact_scores(q, cache, out, lse, scale=None):
    """As check_attention with dz = 0: a score's error is none. The exponents are (s - max) rs in
    f32, a gap g off by at most 2^-21 g (the factors' roundings and the product's), which moves a
    probability by 2^-21 g e^-g < 2^-22, as its ex2.approx does. The log-sum-exp's own size passes
    f32's before the output does: it is infinite there."""
    kc, ks, vc, vs = host(cache)
    b, B, hq, d = q.shape
    qn, on, ln = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = cache.seq_len
    for i in range(min(b, 2)):
        k, v = O.kv4_values(kc[i], ks[i]), O.kv4_values(vc[i], vs[i])
        ref, rl, spread = O.kv4_attention(qn[i], k, v, np.ones(n, bool), scale)
        grid = np.repeat(np.abs(v).sum(1), hq // cache.n_kv_heads, 0) * 2.0 ** -32 + 2.0 ** -133
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + n * 2.0 ** -22) * spread + grid
        assert np.isfinite(on[i]).all()
        assert (np.abs(on[i] - ref) <= tol).all(), (i, np.abs(on[i] - ref).max())
        top = 2.0 ** 128
        sure = np.abs(rl) < top * (1 - 2.0 ** -20)
        assert (np.abs(ln[i] - rl)[sure] <= (n * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(rl)))[sure]).all()
        assert (np.abs(ln[i])[np.abs(rl) > top * (1 + 2.0 ** -20)] == np.inf).all()


@pytest.mark.parametrize("power", [-120, 0, 20, 27, 30, 60, 110, 124])
@pytest.mark.parametrize("b,hq,hkv,d,L,start,B", EXACT_SHAPES)
def test_attention_of_exact_scores(ctx, b, hq, hkv, d, L, start, B, power):
    """Uniform to one-hot rows, with ties, whatever the scores' size."""
    c, q = exact_scores(b, hq, hkv, d, L, B, 161, power)
    out, lse = ctx.kv4_attention(q, c, start, want_lse=True)
    ctx.device_status()
    check_exact_scores(q, c, out, lse)


@pytest.mark.parametrize("scale", [1e-38, 1e30, 3.4e38])
@pytest.mark.parametrize("b,hq,hkv,d,L,start,B", EXACT_SHAPES[2:5])
def test_attention_of_exact_scores_under_any_scale(ctx, b, hq, hkv, d, L, start, B, scale):
    c, q = exact_scores(b, hq, hkv, d, L, B, 162, 0)
    out, lse = ctx.kv4_attention(q, c, start, want_lse=True, scale=scale)
    check_exact_scores(q, c, out, lse, float(np.float32(scale)))


@pytest.mark.parametrize("b,hq,hkv,d,L,B", [
    (1, 32, 32, 128, 768, 32),           # a cluster per unit
    (2, 4, 4, 64, 500, 16),
    (1, 7, 1, 128, 9000, 1),             # clusters of 2 and a join of their parts; rows of one rank
])
def test_a_wait_of_few_rows_that_runs_out_is_reported(b, hq, hkv, d, L, B):
    """The wait for the other blocks' rows follows the context's limit: limited to 1 ns it runs
    out (in one of 20 calls at least: a block may come last), the kernel ends, and the host reads
    FDL_ETIMEOUT; where it did not run out the result is right, and so is a new context's."""
    F = fdl()
    c, q = random_cache(b, hkv, L, d, seed=171), queries(b, B, hq, d, 172)
    x = F.Context(0)
    x.set_wait_timeout(1)
    for _ in range(20):
        out, lse = x.kv4_attention(q, c, 200, want_lse=True)
        try:
            x.device_status()
        except F.FdlError as e:
            assert e.code == F.FDL_ETIMEOUT
            break
        check_attention(q, c, out, lse, 200, seqs=range(1))
    else:
        pytest.fail("no wait ran out")
    x.close()
    torch.cuda.synchronize()
    x = F.Context(0)
    out, lse = x.kv4_attention(q, c, 200, want_lse=True)
    check_attention(q, c, out, lse, 200, seqs=range(1))
    x.device_status()
    x.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_are_the_oracles_bytes(ctx, d, dtype):
    """Under every scale, both signs, with what rounds to 0: a negative value keeps its sign, a
    -0, and whatever is in a group whose scale is 0 or NaN, has none."""
    steps = np.concatenate([[0.0, 1e-30, 0.1, 0.24, 0.25, 0.26, 0.5], np.linspace(0.3, 6, 40)])
    groups = []
    for s in range(1, 127):
        x = np.concatenate([steps, -steps]) * K.E4M3[s]
        x = np.concatenate([x, np.full(-len(x) % 15, -0.0)]).reshape(-1, 15)
        groups.append(np.concatenate([np.full((len(x), 1), -6 * K.E4M3[s]), x], 1))
    tiny = np.resize([-1e-3, 1e-3, -2.0 ** -100, -0.0, 0.0], (5, 16))
    nan = np.resize([-1.0, np.nan, 2.0, -0.0, -np.inf], (5, 16))
    g = np.concatenate(groups + [tiny, -tiny, nan, -nan])
    g = np.concatenate([g, np.full((-len(g) % (d // 16), 16), -0.0)]).reshape(-1, d)
    g = torch.from_numpy(g).to(dtype).double().numpy()
    got, want = store_rows(ctx, g, dtype), O.kv4_quantise(g)
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[0], want[0])
    nib = np.stack((got[0] & 15, got[0] >> 4), -1).reshape(g.shape)
    zero = np.repeat((got[1] == 0) | (got[1] == 127), 16, -1)
    assert zero.any() and (nib[zero | (g == 0)] == 0).all() and (nib[~zero & (g < 0)] >= 8).all()


@pytest.mark.parametrize("hq,hkv,d,L,B", [(4, 4, 128, 600, 32), (8, 2, 64, 500, 7),
                                          (7, 1, 128, 900, 1)])
def test_attention_against_unquantised_rows(ctx, hq, hkv, d, L, B):
    """What the 4 bits cost: with every cached element off by at most 17/96 of its group's largest
    (e_k, e_v), a score moves by at most dz = scale sum |q| e_k, a probability by a factor of at most
    e^(2 dz), so |out - ref| <= sum p e_v + (e^(2 dz) - 1) sum p (|v| + e_v), and the log-sum-exp by dz;
    beside them the kernel's own rounding (here below 2^-6 of sum p |v| and 2^-10)."""
    rng = np.random.default_rng(181)
    k, v = (torch.from_numpy(rng.standard_normal((1, L, hkv, d))).to(torch.bfloat16) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((1, B, hq, d)) / 8).to(torch.bfloat16)
    c = fdl().Kv4Cache.empty(1, hkv, L, d)
    ctx.kv4_store(k.cuda(), v.cuda(), c, 0)
    out, lse = ctx.kv4_attention(q.cuda(), c, 0, want_lse=True)
    qn, kn, vn = (t[0].double().numpy() for t in (q, k, v))
    kn, vn = kn.transpose(1, 0, 2), vn.transpose(1, 0, 2)

    def off(x):
        return np.repeat(np.abs(x).reshape(hkv, L, d // 16, 16).max(-1) * 17 / 96, 16, -1)
    ref, rl, spread = O.kv4_attention(qn, kn, vn, np.ones(L, bool))
    e_v, _, _ = O.kv4_attention(qn, kn, off(vn), np.ones(L, bool))
    # sum p e_v with the probabilities of kn: the values' bounds in the values' place
    dz = np.zeros((B, hq))
    for h in range(hq):
        dz[:, h] = (np.abs(qn[:, h]) @ off(kn)[h // (hq // hkv)].T).max(1) * d ** -0.5
    tol = e_v + np.expm1(2 * dz)[..., None] * (spread + e_v) + 2.0 ** -6 * spread + 2.0 ** -10
    assert (np.abs(out[0].double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse[0].double().cpu().numpy() - rl) <= dz.T + 2.0 ** -10).all()
