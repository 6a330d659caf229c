"""The 4-bit K/V cache without a GPU: the oracle's number formats, and the refusals of the
library's entry points, which come before any device work."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import oracle as O
from block_kv_cache_b200 import fdllm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUP, EWS = fdllm.FDL_EINVAL, fdllm.FDL_EUNSUPPORTED, fdllm.FDL_EWORKSPACE


# ----------------------------------------------------------------- the oracle's formats
def test_e4m3_table_is_torchs():
    t = torch.arange(128, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    from oracle import kv4
    np.testing.assert_array_equal(kv4.E4M3, t)


def test_quantise_ties_and_limits():
    def values(*x):
        row = np.zeros(16)
        row[:len(x)] = x
        return O.kv4_values(*O.kv4_quantise(row))[:len(x)]
    # scale 1 (max 6): every border of two codes goes to the even one
    np.testing.assert_array_equal(
        values(6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -5),
        [6, 0, 1, 1, 2, 2, 4, 4, 0, -4])
    np.testing.assert_array_equal(values(6, .2501, .7499, 2.501, 5.001), [6, .5, .5, 3, 6])
    np.testing.assert_array_equal(values(1e30, -1e30, 448.0), [2688, -2688, 448])
    np.testing.assert_array_equal(values(np.inf, -np.inf, 1.0), [2688, -2688, 0])
    # the scale of a largest value of 3 * 2^-9 is a tie between 0 and 2^-9
    np.testing.assert_array_equal(values(3 * 2.0 ** -9, 2.0 ** -9), [0, 0])
    assert values(3.01 * 2.0 ** -9)[0] == 3 * 2.0 ** -9
    assert np.isnan(O.kv4_values(*O.kv4_quantise(np.array([np.nan] + [1.0] * 15)))).all()


def test_quantise_against_scaled_search():
    """Every value is the nearest product of a code and its group's scale."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((400, 32)) * 2.0 ** rng.integers(-6, 8, (400, 1))
    codes, scales = O.kv4_quantise(x)
    v = O.kv4_values(codes, scales)
    from oracle import kv4
    s = np.repeat(kv4.E4M3[scales], 16, -1)
    grid = np.concatenate([-kv4.E2M1, kv4.E2M1])
    best = np.abs(x[..., None] - grid * s[..., None]).min(-1)
    np.testing.assert_array_equal(np.abs(x - v), best)


def test_visible_positions():
    v = O.kv4_visible(20, 8, 4, 18, (3, 2), 2)
    assert np.flatnonzero(v).tolist() == [0, 1] + list(range(5, 14))
    assert O.kv4_visible(20, 8, 4, 9, (3, 2), 2).sum() == 2 + 4
    assert O.kv4_visible(20, 8, 4, 0).sum() == 0
    assert O.kv4_visible(20, 8, 4).sum() == 20
    assert np.flatnonzero(O.kv4_visible(20, 0, 1, None, (0, 0), 5)).tolist() == [0, 1, 2, 3, 4]


# ------------------------------------------------------------------------ the binding
def _header():
    return open(os.path.join(ROOT, "include", "fdllm.h")).read()


def test_structs_match_the_header():
    sizes = {"int": 4, "float": 4, "int64_t": 8}
    for cname, py in (("fdl_kv4_cache", fdllm.Kv4Buffers),
                      ("fdl_kv4_rows_desc", fdllm.Kv4RowsDesc),
                      ("fdl_kv4_attn_desc", fdllm.Kv4AttnDesc)):
        src = _header()
        end = re.search(r"\}\s*" + cname + r"\s*;", src).start()
        body = re.sub(r"/\*.*?\*/", "", src[src.rindex("typedef struct {", 0, end):end]
                      .split("{", 1)[1], flags=re.S)
        fields = re.findall(r"([\w\s\*]+?)\s*\b(\w+);", body)
        assert [f for _, f in fields] == [f for f, _ in py._fields_], cname
        for (ctype, fname), (_, pytype) in zip(fields, py._fields_):
            assert ctypes.sizeof(pytype) == (8 if "*" in ctype else sizes[ctype.strip()]), fname


# ------------------------------------------------------------------- refusals, no device
# A context is only looked into once every argument has passed: zeroed memory
# stands in for one. Addresses are never followed.
CTX = ctypes.create_string_buffer(4096)
ctypes.cast(CTX, ctypes.POINTER(ctypes.c_int))[1] = 148      # its SM count
P = 1 << 20                                                  # an aligned "address"


def ctx():
    return ctypes.cast(CTX, ctypes.c_void_p)


def cache(**kw):
    b = fdllm.Kv4Buffers(P, P, P, P)
    for k, v in kw.items():
        setattr(b, k, v)
    return ctypes.byref(b)


def rows(**kw):
    f = dict(batch=2, n_kv_heads=4, head_dim=128, seq_len=100, dtype=fdllm.FDL_BF16,
             seq_stride=0, row_stride=0, head_stride=0)
    f.update(kw)
    return ctypes.byref(fdllm.Kv4RowsDesc(**f))


BAD_ROWS = [
    (dict(batch=0), EINVAL), (dict(batch=65536), EINVAL), (dict(n_kv_heads=0), EINVAL),
    (dict(seq_len=0), EINVAL), (dict(head_dim=96), EUNSUP), (dict(head_dim=32), EUNSUP),
    (dict(dtype=2), EINVAL), (dict(row_stride=-8), EINVAL),
    (dict(row_stride=516, head_stride=128, seq_stride=51200), EINVAL),
    (dict(seq_len=(1 << 30) + 1), EUNSUP), (dict(seq_len=2147483647), EUNSUP),
]


@pytest.mark.parametrize("kw,code", BAD_ROWS)
def test_store_and_load_refuse_bad_descriptors(kw, code):
    L = fdllm.load()
    assert L.fdl_kv4_store(ctx(), rows(**kw), P, P, 0, 10, cache(), None) == code
    assert L.fdl_kv4_load(ctx(), rows(**kw), cache(), 0, 10, P, P, None) == code
    assert len(L.fdl_last_error()) > 0


@pytest.mark.parametrize("start,n", [(0, 0), (0, -1), (-1, 5), (91, 10), (0, 101),
                                     (2147483647, 1), (1, 2147483647)])
def test_store_and_load_refuse_bad_ranges(start, n):
    L = fdllm.load()
    assert L.fdl_kv4_store(ctx(), rows(), P, P, start, n, cache(), None) == EINVAL
    assert L.fdl_kv4_load(ctx(), rows(), cache(), start, n, P, P, None) == EINVAL


def test_store_and_load_refuse_bad_buffers():
    L = fdllm.load()
    assert L.fdl_kv4_store(None, rows(), P, P, 0, 10, cache(), None) == EINVAL
    assert L.fdl_kv4_store(ctx(), None, P, P, 0, 10, cache(), None) == EINVAL
    assert L.fdl_kv4_store(ctx(), rows(), None, P, 0, 10, cache(), None) == EINVAL
    assert L.fdl_kv4_store(ctx(), rows(), P, None, 0, 10, cache(), None) == EINVAL
    assert L.fdl_kv4_store(ctx(), rows(), P + 8, P, 0, 10, cache(), None) == EINVAL
    assert L.fdl_kv4_store(ctx(), rows(), P, P, 0, 10, None, None) == EINVAL
    for f in ("k", "k_scale", "v", "v_scale"):
        assert L.fdl_kv4_store(ctx(), rows(), P, P, 0, 10, cache(**{f: None}), None) == EINVAL
        assert L.fdl_kv4_load(ctx(), rows(), cache(**{f: P + 4}), 0, 10, P, P, None) == EINVAL
    assert L.fdl_kv4_load(ctx(), rows(), cache(), 0, 10, None, None, None) == EINVAL
    assert L.fdl_kv4_load(ctx(), rows(), cache(), 0, 10, P + 2, P, None) == EINVAL
    # rows written on top of one another
    same = dict(head_stride=128, row_stride=0, seq_stride=5120)
    assert L.fdl_kv4_load(ctx(), rows(**same), cache(), 0, 10, P, P, None) == EINVAL
    # more heads than one call's grid holds
    assert L.fdl_kv4_store(ctx(), rows(n_kv_heads=32768), P, P, 0, 9, cache(), None) == EUNSUP


def attn(**kw):
    f = dict(batch=2, n_q_heads=8, n_kv_heads=4, head_dim=128, seq_len=100, block_start=50,
             block_len=32, dtype=fdllm.FDL_BF16, scale=0.0, window_left=-1, window_right=-1,
             sinks=0)
    f.update(kw)
    return ctypes.byref(fdllm.Kv4AttnDesc(**f))


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), EINVAL), (dict(n_q_heads=6), EINVAL), (dict(n_kv_heads=0), EINVAL),
    (dict(head_dim=96), EUNSUP), (dict(dtype=fdllm.FDL_F32), EUNSUP), (dict(dtype=7), EINVAL),
    (dict(block_len=0), EINVAL), (dict(block_len=129, seq_len=400), EINVAL),
    (dict(block_start=-1), EINVAL), (dict(block_start=69), EINVAL),
    (dict(block_start=2147483647), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(sinks=-1), EINVAL), (dict(batch=1 << 22, n_q_heads=64), EUNSUP),
    (dict(seq_len=(1 << 30) + 1), EUNSUP), (dict(seq_len=2147483647, block_start=2147483615), EUNSUP),
])
def test_attention_refuses_bad_descriptors(kw, code):
    L = fdllm.load()
    assert L.fdl_kv4_attention(ctx(), attn(**kw), P, cache(), None, 2 * P, None, P, 1 << 40,
                               None) == code
    assert L.fdl_kv4_attention_workspace_bytes(ctx(), attn(**kw)) == 0


def test_attention_refuses_bad_buffers():
    L = fdllm.load()

    def call(c=None, d=None, q=P, ca=None, kv_len=None, out=2 * P, lse=None, ws=P, n=1 << 30):
        return L.fdl_kv4_attention(c or ctx(), d or attn(), q, ca or cache(), kv_len, out, lse, ws,
                                   n, None)
    assert L.fdl_kv4_attention(None, attn(), P, cache(), None, 2 * P, None, P, 99, None) == EINVAL
    assert L.fdl_kv4_attention(ctx(), None, P, cache(), None, 2 * P, None, P, 99, None) == EINVAL
    assert L.fdl_kv4_attention(ctx(), attn(), P, None, None, 2 * P, None, P, 99, None) == EINVAL
    assert call(q=None) == EINVAL
    assert call(out=None) == EINVAL
    assert call(out=P) == EINVAL                             # in place
    assert call(q=P + 8) == EINVAL
    assert call(out=2 * P + 8) == EINVAL
    assert call(lse=P + 2) == EINVAL
    assert call(kv_len=P + 1) == EINVAL
    assert call(ca=cache(v_scale=None)) == EINVAL
    assert call(ca=cache(k_scale=P + 8)) == EINVAL
    # one token of a long sequence: split widely, with partial results
    long = attn(batch=1, seq_len=1 << 20, block_len=1)
    need = L.fdl_kv4_attention_workspace_bytes(ctx(), long)
    assert need > 16
    assert call(d=long, ws=None) == EWS
    assert call(d=long, ws=P + 4) == EWS
    assert call(d=long, n=need - 1) == EWS
    assert L.fdl_kv4_attention_workspace_bytes(ctx(), attn()) == 16      # none, and none asked for
    assert L.fdl_kv4_attention_workspace_bytes(None, attn()) == 0
    # widths beyond int: the window is clipped to the sequence, not wrapped
    assert L.fdl_kv4_attention_workspace_bytes(
        ctx(), attn(window_left=2147483647, window_right=2147483647, sinks=2147483647)) > 0


def test_binding_refuses_cpu_tensors():
    z = torch.zeros((1, 1, 4, 64), dtype=torch.uint8)
    s = torch.zeros((1, 1, 4, 8), dtype=torch.uint8)
    with pytest.raises(TypeError):
        fdllm.Kv4Cache(z, s, z, s)


def test_binding_refuses_what_ctypes_would_cut():
    """Numbers beyond 32 bits are errors, not their lower halves."""
    import types
    c = types.SimpleNamespace(batch=1, n_kv_heads=2, seq_len=100, head_dim=64, device_index=0)
    x = fdllm.Context.__new__(fdllm.Context)
    x.device, x._h, x._kv4_descs = 0, None, {}
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    big = 1 << 32
    assert x.kv4_attn_desc(q, c, 8, (3, 5), 2).window_right == 5
    for at, window, sinks in ((big, (-1, -1), 0), (0, (big + 4, 0), 0), (0, (0, big), 0),
                              (0, (-1, -1), big), (0, (-1, -(1 << 31) - 1), 0)):
        with pytest.raises(ValueError):
            x.kv4_attn_desc(q, c, at, window, sinks)
    with pytest.raises(ValueError):
        x.kv4_attn_desc(q, c, -big)
    with pytest.raises(ValueError):
        x.kv4_load(c, big)
    with pytest.raises(ValueError):
        x.kv4_load(c, 0, big + 1)
    # a stream of another device
    other = types.SimpleNamespace(device_index=1)
    for call in (lambda: x.kv4_load(c, stream=other), lambda: x.kv4_store(q, q, c, 0, stream=other),
                 lambda: x.kv4_attention(q, c, 0, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


class Recorder:
    """Stands in for the library: keeps what the attention was called with."""

    def __init__(self, need=16):
        self.calls, self.need = [], need

    def fdl_kv4_attention(self, h, desc, q, cache, kv_len, out, lse, ws, ws_bytes, stream):
        d = desc._obj
        self.calls.append((d.block_start, d.window_left, d.window_right, d.sinks, d.scale))
        return 0

    def fdl_kv4_attention_workspace_bytes(self, h, desc):
        return self.need


def host_context(monkeypatch, lib):
    """A context whose calls go to `lib` with CPU tensors, and a cache for it."""
    import types
    monkeypatch.setattr(fdllm, "_lib", lib)
    monkeypatch.setattr(fdllm, "_raw_stream", lambda device: 0)
    x = fdllm.Context.__new__(fdllm.Context)
    x.device, x._h, x._kv4_descs, x._seeds = -1, None, {}, {}
    c = types.SimpleNamespace(batch=1, n_kv_heads=2, seq_len=100, head_dim=64, device_index=-1,
                              buffers=fdllm.Kv4Buffers())
    return x, c, torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)


def test_arguments_are_read_at_every_call(monkeypatch):
    """Tensors as numbers, changed in place between two calls."""
    lib = Recorder()
    x, c, q = host_context(monkeypatch, lib)
    start, left, right, sinks = (torch.tensor(v) for v in (8, 5, 6, 4))
    scale = torch.tensor(0.5)
    x.kv4_attention(q, c, start, window=(left, right), sinks=sinks, scale=scale)
    for t in (left, right, sinks):
        t += 10
    scale += 0.5
    x.kv4_attention(q, c, start, window=(left, right), sinks=sinks, scale=scale)
    assert lib.calls == [(8, 5, 6, 4, 0.5), (8, 15, 16, 14, 1.0)]
    start += 10
    x.kv4_attention(q, c, start, window=(left, right), sinks=sinks, scale=scale)
    assert lib.calls[2:] == [(18, 15, 16, 14, 1.0)]


@pytest.mark.parametrize("b,h,n,strides,ok", [
    (2, 4, 10, (5120, 512, 128), True),                      # [b, n, Hkv, d]
    (2, 4, 10, (5120, 128, 1280), True),                     # [b, Hkv, n, d]
    (2, 4, 10, (128, 256, 2560), True),                      # [Hkv, n, b, d]
    (2, 4, 10, (10000, 136, 1600), True),                    # with room between
    (2, 4, 10, (1 << 61, 1 << 55, 1 << 50), True),
    (1, 1, 10, (0, 128, 0), True),                           # a single one has no stride
    (2, 4, 10, (5120, 128, 128), False),                     # row on row of the next head
    (2, 4, 10, (8, 512, 128), False),                        # sequences 8 elements apart
    (2, 4, 10, (5120 - 8, 512, 128), False),
    (2, 4, 10, (5120, 504, 128), False),
    (2, 4, 10, (5120, 512, 120), False),
    (2, 4, 10, (5120, 128, 1272), False),
    (2, 1, 10, (0, 128, 0), False),
])
def test_load_refuses_rows_that_overlap(monkeypatch, b, h, n, strides, ok):
    """What passes the check goes on to the device, of which there is none here; the places of
    the rows, where they can be listed, agree."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    L = fdllm.load()
    d = rows(batch=b, n_kv_heads=h, seq_stride=strides[0], row_stride=strides[1],
             head_stride=strides[2])
    rc = L.fdl_kv4_load(ctx(), d, cache(), 0, n, P, 1 << 45, None)
    assert rc == (fdllm.FDL_ECUDA if ok else EINVAL)
    assert ok == (b"overlap" not in L.fdl_last_error())
    if max(strides) < 1 << 20:
        at = np.add.outer(np.add.outer(np.arange(b) * strides[0], np.arange(n) * strides[1]),
                          np.arange(h) * strides[2]).ravel()[:, None] + np.arange(128)
        assert ok == (len(np.unique(at)) == at.size)


def _places(b, h, n, strides, d=64):
    return (np.add.outer(np.add.outer(np.arange(b) * strides[0], np.arange(n) * strides[1]),
                         np.arange(h) * strides[2]).ravel()[:, None] + np.arange(d)).ravel()


def test_load_refuses_k_and_v_on_top_of_one_another():
    """K's and V's rows interleaved in one buffer in every way, and the ways that overlap: refused
    exactly where a place occurs in both."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    L = fdllm.load()
    rng = np.random.default_rng(5)
    seen = {True: 0, False: 0}
    for _ in range(1500):
        b, h, n = (int(x) for x in rng.integers(1, 4, 3))
        strides, span = [0, 0, 0], 64
        for i in rng.permutation(3):
            strides[i] = span + 8 * int(rng.choice([0, 0, 1, 8, 24, 9 * int(rng.integers(1, 8))]))
            span = strides[i] * (b, n, h)[i]
        delta = 8 * int(rng.integers(-span // 8 - 20, span // 8 + 21))
        at = _places(b, h, n, strides)
        ok = not np.intersect1d(at, at + delta).size
        d = rows(batch=b, n_kv_heads=h, head_dim=64, seq_stride=strides[0], row_stride=strides[1],
                 head_stride=strides[2])
        k = 1 << 40
        rc = L.fdl_kv4_load(ctx(), d, cache(), 0, n, k, k + 2 * delta, None)
        assert rc == (fdllm.FDL_ECUDA if ok else EINVAL), (b, h, n, strides, delta)
        seen[ok] += 1
    assert min(seen.values()) > 300
    assert L.fdl_kv4_load(ctx(), rows(), cache(), 0, 10, P, P, None) == EINVAL
    assert L.fdl_kv4_load(ctx(), rows(), cache(), 0, 10, P, P + 100 * 1024, None) == fdllm.FDL_ECUDA


def test_attention_refuses_out_that_overlaps_q():
    L = fdllm.load()
    d, size, q = attn(), 2 * 32 * 8 * 128 * 2, 1 << 40
    for delta in (0, 16, -16, size - 16, 16 - size):
        assert L.fdl_kv4_attention(ctx(), d, q, cache(), None, q + delta, None, P, 1 << 30,
                                   None) == EINVAL
    assert b"overlap" in L.fdl_last_error()
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for delta in (size, -size):
        assert L.fdl_kv4_attention(ctx(), d, q, cache(), None, q + delta, None, P, 1 << 30,
                                   None) == fdllm.FDL_ECUDA


def test_quantise_signs_of_zeros():
    x = np.resize([6.0, -0.1, 0.1, -0.0, 0.0, -1.0], 16)
    codes, _ = O.kv4_quantise(x)
    nib = np.stack((codes & 15, codes >> 4), -1).ravel()
    np.testing.assert_array_equal(nib, np.resize([7, 8, 0, 0, 0, 10], 16))
    for y in (x * 1e-4, np.concatenate([x[:15], [np.nan]])):               # scales 0 and NaN
        codes, scale = O.kv4_quantise(y)
        assert scale[0] in (0, 127) and not codes.any()


def test_plan_query():
    """What the query says of both kernels' shapes on 148 SMs, and its refusals."""
    L = fdllm.load()

    def plan(**kw):
        p = fdllm.Kv4Plan()
        assert L.fdl_kv4_attention_plan(ctx(), attn(**kw), ctypes.byref(p)) == 0
        return p
    p = plan(batch=1, seq_len=1 << 20, block_len=1)
    assert (p.many_rows, p.row_tiles, p.cluster) == (0, 1, 2) and p.splits > 8
    assert plan().many_rows == 0 and plan().row_tiles == 2
    p = plan(batch=32, n_q_heads=28, seq_len=1024)
    assert (p.many_rows, p.row_tiles, p.splits, p.cluster) == (1, 2, 1, 1)
    assert L.fdl_kv4_attention_plan(None, attn(), ctypes.byref(p)) == EINVAL
    assert L.fdl_kv4_attention_plan(ctx(), attn(), None) == EINVAL
    assert L.fdl_kv4_attention_plan(ctx(), None, ctypes.byref(p)) == EINVAL
    assert L.fdl_kv4_attention_plan(ctx(), attn(head_dim=96), ctypes.byref(p)) == EUNSUP
    body = re.search(r"typedef struct \{([^}]*)\} fdl_kv4_plan;", _header()).group(1)
    assert re.findall(r"int (\w+);", body) == [f for f, _ in fdllm.Kv4Plan._fields_]


def test_scratch_is_asked_for_once_and_without_an_error(monkeypatch):
    """A shape's scratch is known before its first call: one call reaches the library, and none
    that is refused (whose text would stay behind as the last error)."""
    for need in (16, 4096):
        lib = Recorder(need)
        sizes, asked = [], []
        lib.fdl_kv4_attention = lambda *a: sizes.append((a[7] is not None, a[8])) or \
            (EWS if a[8] < need and need > 16 else 0)
        lib.fdl_kv4_attention_workspace_bytes = lambda *a: asked.append(1) or need
        x, c, q = host_context(monkeypatch, lib)
        x._seeds[torch.uint8] = torch.empty(0, dtype=torch.uint8)
        for _ in range(3):
            x.kv4_attention(q, c, 8)
        assert sizes == 3 * [(need > 16, need if need > 16 else 0)]
        assert len(asked) == 1


def test_a_caches_tensors_are_not_replaced():
    """The calls go to the addresses that the cache was made with."""
    c = fdllm.Kv4Cache.__new__(fdllm.Kv4Cache)
    c._tensors = tuple(torch.full((1,), i) for i in range(4))
    for i, name in enumerate(("k", "k_scale", "v", "v_scale")):
        assert getattr(c, name) is c._tensors[i]
        with pytest.raises(AttributeError):
            setattr(c, name, torch.zeros(1))


def test_store_refuses_a_cache_on_top_of_itself():
    """K's and V's rows are written at once: their codes and scales lie apart."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    L = fdllm.load()
    codes, scales, at = 2 * 4 * 100 * 64, 2 * 4 * 100 * 8, 1 << 40

    def store(k, ks, v, vs):
        return L.fdl_kv4_store(ctx(), rows(), P, P, 0, 10,
                               cache(k=at + k, k_scale=at + ks, v=at + v, v_scale=at + vs), None)
    apart = (0, codes, codes + scales, 2 * codes + scales)
    assert store(*apart) == store(apart[2], apart[3], apart[0], apart[1]) == fdllm.FDL_ECUDA
    for bad in ((0, 2 * codes, 0, 3 * codes), (0, 2 * codes, codes, 2 * codes),
                (0, 2 * codes, codes - 16, 3 * codes), (codes - 16, 2 * codes, 0, 3 * codes),
                (0, codes, 2 * codes, codes + scales - 16), (0, codes - 16, 2 * codes, 3 * codes),
                (16, 0, 2 * codes, 3 * codes)):
        assert store(*bad) == EINVAL
        assert b"overlap" in L.fdl_last_error()


@pytest.mark.parametrize("d,hq,b,hkv,below,above", [
    (128, 32, 1, 8, 3900, 4000), (128, 28, 1, 4, 9700, 9800),            # edges 850 and 1850
    (64, 32, 4, 8, 1700, 1800), (64, 28, 4, 4, 3400, 3500),              # 1500 and 2600
])
def test_the_plan_changes_kernels_where_it_was_measured(d, hq, b, hkv, below, above):
    L = fdllm.load()

    def many(n, **kw):
        p = fdllm.Kv4Plan()
        assert L.fdl_kv4_attention_plan(ctx(), attn(batch=b, n_q_heads=hq, n_kv_heads=hkv,
                                                    head_dim=d, seq_len=n, **kw), ctypes.byref(p)) == 0
        return p.many_rows
    assert (many(below), many(above)) == (0, 1)
    assert many(1 << 20, window_left=20, window_right=0) == 0            # what is seen counts


def test_quantisation_error_is_the_documented_one():
    """With scale = (max / 6)(1 + e), |e| <= 2^-4, a quotient is at most 6 / (1 - 2^-4) = 6.4 and
    its code off by at most 1 (between 4 and 6; 0.4 beyond 6): scale <= 17/96 max. A subnormal
    scale is off by up to 2^-10, which a code of 6 multiplies."""
    rng = np.random.default_rng(3)
    for exponent in range(-14, 12):
        x = rng.standard_normal((2000, 16)) * 2.0 ** exponent * rng.uniform(0.5, 1, (2000, 1))
        x = np.concatenate([x, rng.uniform(-1, 1, (2000, 16)) * 2.0 ** exponent])
        x = np.clip(x, -2688, 2688)
        err = np.abs(O.kv4_values(*O.kv4_quantise(x)) - x).max(1)
        top = np.abs(x).max(1)
        bound = np.where(top >= 6 * 2.0 ** -6, top * 17 / 96,
                         np.maximum(top / 6 + 2.0 ** -10, 6 * 2.0 ** -10))
        assert (err <= bound * (1 + 1e-12)).all(), exponent
        if -3 < exponent < 8:
            rel = np.linalg.norm(O.kv4_values(*O.kv4_quantise(x[:2000])) - x[:2000])
            assert 0.08 < rel / np.linalg.norm(x[:2000]) < 0.10
