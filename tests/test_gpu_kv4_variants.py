"""Every form of the attention over the 4-bit K/V cache (both kernels, one and two tiles of rows,
both head sizes, units of rows alone in a block, joined over a cluster, and joined in the
workspace too) under every property that a call may have: lengths, windows and first positions,
NaN in what is not seen, sizes of queries, maxima that grow, captured and replayed. What a shape
is for is checked against the library's plan, so that a changed rule cannot move the cases to
another form unseen. Tolerances as in test_gpu_kv4.py."""
from collections import namedtuple

import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_kv4 import check_attention, fdl, queries

pytestmark = pytest.mark.gpu

V = namedtuple("V", "many tiles join d b hq hkv L start B")
VARIANTS = [
    V(many, tiles, join, d, *shape) for d in (64, 128) for many, tiles, join, shape in [
        # b, Hq, Hkv, L, start, B
        (1, 2, "alone", (19, 28, 4, 190, 101, 32)),      # 224 rows
        (1, 1, "alone", (19, 20, 4, 190, 101, 17)),      # 85
        (1, 2, "cluster", (6, 28, 4, 700, 411, 32)),     # 224, 24 units
        (1, 1, "cluster", (10, 16, 4, 700, 411, 31)),    # 124, 40 units
        (1, 2, "parts", (2, 64, 8, 6300, 3300, 31)),     # 248, 16 units
        (1, 1, "parts", (4, 16, 4, 7300, 4100, 31)),     # 124, 16 units
        (0, 2, "alone", (19, 8, 8, 190, 101, 29)),       # 29
        (0, 1, "alone", (19, 16, 8, 190, 101, 7)),       # 14
        (0, 2, "cluster", (5, 12, 4, 700, 411, 9)),      # 27
        (0, 1, "cluster", (5, 24, 8, 700, 411, 5)),      # 15
        (0, 2, "parts", (2, 4, 4, 2300, 1300, 32)),      # 32
        (0, 1, "parts", (2, 7, 1, 2300, 2299, 1)),       # a token, 7
    ]]


@pytest.fixture(scope="module")
def ctx():
    c = fdl().Context(0)
    yield c
    c.close()


@pytest.fixture(scope="module", params=VARIANTS, ids=lambda v: "-".join(map(str, v)))
def case(request, ctx):
    v = request.param
    g = torch.Generator(device="cuda").manual_seed(7)
    c = fdl().Kv4Cache.empty(v.b, v.hkv, v.L, v.d)
    big = torch.where(torch.rand(v.d, generator=g, device="cuda") > 0.94, 6.0, 0.7)
    k, x = (torch.randn((v.b, v.L, v.hkv, v.d), generator=g, device="cuda") for _ in range(2))
    ctx.kv4_store(k * big, x, c, 0)
    return v, c


def attend(ctx, v, q, c, **kw):
    """The call, after a look at how the library runs it."""
    p = ctx.kv4_attention_plan(ctx.kv4_attn_desc(q, c, v.start, kw.get("window", (-1, -1)),
                                                 kw.get("sinks", 0)))
    join = "alone" if p.splits == 1 else "cluster" if p.splits == p.cluster else "parts"
    assert (p.many_rows, p.row_tiles, join) == (v.many, v.tiles, v.join)
    out, lse = ctx.kv4_attention(q, c, v.start, want_lse=True, **kw)
    ctx.device_status()
    return out, lse


def lengths(v, kinds):
    n = [kinds[i % len(kinds)] for i in range(v.b)]
    return n, torch.tensor(n, dtype=torch.int32, device="cuda")


def copy_of(c):
    return fdl().Kv4Cache(*(t.clone() for t in (c.k, c.k_scale, c.v, c.v_scale)))


def test_lengths(ctx, case):
    """None, one, part of a step, a whole number of steps, all, and beyond either end."""
    v, c = case
    q = queries(v.b, v.B, v.hq, v.d, 2)
    for kinds in ((0, 1, v.L // 2 + 3, v.L + 1000, -7), (64, 16, 65, 2, v.L - 1), (0,)):
        n, t = lengths(v, kinds)
        out, lse = attend(ctx, v, q, c, kv_len=t)
        check_attention(q, c, out, lse, v.start, [max(0, min(v.L, x)) for x in n],
                        seqs=range(min(v.b, 5)))


def near(v):
    """Positions before the block that a window shows, enough for the variant's splits."""
    return {"alone": 61, "cluster": 200, "parts": v.L // 2}[v.join]


def test_windows_and_first_positions(ctx, case):
    """A gap behind the first positions, none, one of nothing, and lengths that end before the
    window, inside it, and among the first positions."""
    v, c = case
    q = queries(v.b, v.B, v.hq, v.d, 3)
    for window, sinks in (((near(v), v.L // 8), 3), ((near(v), v.L // 8), 0),
                          ((v.start - 5, 0), 5), ((v.start - 40, -1), 33)):
        n, t = lengths(v, (v.L, v.start + v.B // 2, 2, v.start - 3, v.start + v.B + 1))
        out, lse = attend(ctx, v, q, c, kv_len=t, window=window, sinks=sinks)
        check_attention(q, c, out, lse, v.start, n, window, sinks, seqs=range(min(v.b, 5)))


def test_nothing_seen(ctx, case):
    """Every sequence ends before its window, and there are no first positions."""
    v, c = case
    q = queries(v.b, v.B, v.hq, v.d, 4)
    _, t = lengths(v, (v.start - near(v),))
    out, lse = attend(ctx, v, q, c, kv_len=t, window=(near(v), v.L // 8))
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_what_is_not_seen_may_hold_anything(ctx, case):
    v, c = case
    q = queries(v.b, v.B, v.hq, v.d, 5)
    window, sinks = (near(v), 21), 3
    n, t = lengths(v, (v.L - 37, v.start + 5, 1, 0))
    clean = attend(ctx, v, q, c, kv_len=t, window=window, sinks=sinks)
    d = copy_of(c)
    for i in range(v.b):
        unseen = torch.from_numpy(~O.kv4_visible(v.L, v.start, v.B, n[i], window, sinks)).cuda()
        for x in (d.k, d.k_scale, d.v, d.v_scale):
            x[i][:, unseen] = 0x7f if x.shape[-1] == v.d // 16 else 0xff
    dirty = attend(ctx, v, q, d, kv_len=t, window=window, sinks=sinks)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_nan_reaches_only_what_sees_it(ctx, case):
    v, c = case
    d, q = copy_of(c), queries(v.b, v.B, v.hq, v.d, 6)
    G, last = v.hq // v.hkv, v.hkv - 1
    d.v_scale[1, last, v.L - 2, 2] = 127        # a value of the last kv head: dims 32..47
    out, lse = attend(ctx, v, q, d)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, :, last * G:, 32:48] = True
    assert torch.equal(torch.isnan(out), bad) and not torch.isnan(lse).any()
    d.k_scale[0, 0, v.L // 2, 3] = 127          # a key of the first
    out, lse = attend(ctx, v, q, d)
    bad[0, :, :G] = True
    rows = torch.zeros_like(lse, dtype=torch.bool)
    rows[0, :G] = True
    assert torch.equal(torch.isnan(out), bad) and torch.equal(torch.isnan(lse), rows)


@pytest.mark.parametrize("size", [2.0 ** -126, 1e-3, 30.0])
def test_query_sizes(ctx, case, size):
    v, c = case
    q = queries(v.b, v.B, v.hq, v.d, 8, size)
    out, lse = attend(ctx, v, q, c)
    check_attention(q, c, out, lse, v.start, seqs=(0, v.b - 1))


def test_query_rows_of_mixed_sizes(ctx, case):
    """Rows, and elements within a row, many powers of two apart; a row of zeros."""
    v, c = case
    q = queries(v.b, v.B, v.hq, v.d, 9).float()
    q = q * torch.exp2(torch.arange(v.B, device="cuda") % 13 - 9.0)[:, None, None] \
        * torch.exp2(-(torch.arange(v.d, device="cuda") % 20.0))
    q[:, v.B // 2, 0] = 0
    q = q.to(torch.bfloat16)
    out, lse = attend(ctx, v, q, c, scale=0.5)
    check_attention(q, c, out, lse, v.start, scale=0.5, seqs=(0, v.b - 1))


def test_scores_that_grow_along_the_sequence(ctx, case):
    """The running maximum is raised again and again."""
    v, _ = case
    g = torch.Generator(device="cuda").manual_seed(10)
    u = torch.randn(v.d, generator=g, device="cuda")
    k, x = (torch.randn((v.b, v.L, v.hkv, v.d), generator=g, device="cuda") for _ in range(2))
    k += torch.linspace(-20, 20, v.L, device="cuda")[:, None, None] * u
    c = fdl().Kv4Cache.empty(v.b, v.hkv, v.L, v.d)
    ctx.kv4_store(k, x, c, 0)
    q = (u + torch.randn((v.b, v.B, v.hq, v.d), generator=g, device="cuda")) / 4
    q = q.to(torch.bfloat16)
    out, lse = attend(ctx, v, q, c)
    check_attention(q, c, out, lse, v.start, seqs=(0, v.b - 1))


def test_captured_and_replayed(ctx, case):
    """Two graphs of one form in turn, with other queries, rows and lengths each time."""
    v, c0 = case
    graphs = []
    for i in range(2):
        c, q = copy_of(c0), queries(v.b, v.B, v.hq, v.d, 11 + i)
        _, t = lengths(v, (v.L,))
        rows = queries(v.b, v.B, v.hkv, v.d, 13 + i)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ctx.kv4_attention(q, c, v.start, kv_len=t)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.kv4_store(rows, rows, c, v.start)
            out, lse = ctx.kv4_attention(q, c, v.start, kv_len=t, want_lse=True)
        graphs.append((g, c, q, t, rows, out, lse))
    for r in range(2):
        for i in (1, 0):
            g, c, q, t, rows, out, lse = graphs[i]
            q.copy_(queries(v.b, v.B, v.hq, v.d, 20 + r))
            rows.copy_(queries(v.b, v.B, v.hkv, v.d, 30 + r))
            n, new = lengths(v, (v.L - r, 0 if r else 37, v.start + v.B))
            t.copy_(new)
            g.replay()
            torch.cuda.synchronize()
            check_attention(q, c, out, lse, v.start, n, seqs=range(min(v.b, 2)))
    ctx.device_status()


def test_two_calls_at_once(ctx, case):
    """Two streams' calls, each with its own scratch, and a store between, do not disturb one
    another."""
    v, c = case
    cs, qs = [copy_of(c) for _ in range(2)], [queries(v.b, v.B, v.hq, v.d, 41 + i) for i in range(2)]
    rows = [queries(v.b, v.B, v.hkv, v.d, 43 + i) for i in range(2)]
    streams, got, want = [torch.cuda.Stream() for _ in range(2)], [[], []], []
    for i in range(2):
        ctx.kv4_store(rows[i], rows[i], cs[i], v.start)
        want.append(attend(ctx, v, qs[i], cs[i]))
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            ctx.kv4_store(rows[i], rows[i], cs[i], v.start, stream=streams[i])
            got[i].append(ctx.kv4_attention(qs[i], cs[i], v.start, want_lse=True,
                                            stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    ctx.device_status()
