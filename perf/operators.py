"""Measured cases of the 4-bit K/V cache: writing it, reading it back, and the block
attention that reads it.

The cache holds keys and values in microscaled 4-bit floating point. Along head_dim, every
group of 16 values shares one scale:
  scale = e4m3(max |x| / 6)   (round to nearest even, at most 448; 8 bits)
  code  = e2m1(x / scale)     (round to nearest even, saturating at 6; 4 bits; 0 where scale = 0)
and stands for code * scale. Layouts: codes [b, Hkv, L, d/2] uint8 (the even dimension of a
pair in the low nibble), scales [b, Hkv, L, d/16] uint8, K and V apart.

A case is one of
  "write": n fresh rows of every sequence, quantised into the cache, then read back from it
  "read":  n rows of every sequence, read back from the cache
  "attend": the block's queries over the cache, softmax over the visible positions j:
            j < kv_len[sequence], and j < sinks or
            block_start - left <= j < block_start + block + right   (left, right < 0: no bound)
            with the output and the log-sum-exp; nothing visible gives 0 and -inf
"""
import math

import torch

own = False

GROUP = 16
FDL_SCALE = {64: 0.125, 128: 128 ** -0.5}


# ------------------------------------------------------------------------- cases
def _write(name, b, hkv, d, L, start, n, dtype="bf16", order="token"):
    return {"name": name, "op": "write", "b": b, "hkv": hkv, "d": d, "L": L, "start": start,
            "n": n, "dtype": dtype, "order": order}


def _read(name, b, hkv, d, L, start, n, dtype="bf16"):
    return {"name": name, "op": "read", "b": b, "hkv": hkv, "d": d, "L": L, "start": start,
            "n": n, "dtype": dtype}


def _attend(name, b, hq, hkv, d, L, start, block, lens="full", left=-1, right=-1, sinks=0):
    return {"name": name, "op": "attend", "b": b, "hq": hq, "hkv": hkv, "d": d, "L": L,
            "start": start, "block": block, "lens": lens, "left": left, "right": right,
            "sinks": sinks}


def listed():
    return [
        # one block of a cached step of the 32-head model, prompt 512 + 256 generated
        _write("write_block", 1, 32, 128, 768, 512, 32),
        # its refresh at 2048 positions: every row of a layer
        _write("write_refresh", 1, 32, 128, 2048, 0, 2048),
        # the refresh of a batch of 32 with 4 kv heads, from a layer's head-major bf16 rows
        _write("write_batch32_heads_first", 32, 4, 128, 1024, 0, 1024, order="head"),
        # f32 rows of an odd range, 64-dim heads
        _write("write_f32_odd", 3, 2, 64, 1003, 37, 517, dtype="f32"),
        # the cached prompts of the batch of 32, for a step that recomputes the rest
        _read("read_prefix_batch32", 32, 4, 128, 1024, 0, 512),
        # nearly all of an odd cache, as f32
        _read("read_f32_odd", 3, 8, 64, 4099, 1, 4097, dtype="f32"),
        # a cached step's attention, prompt 512 + 256 generated
        _attend("attend_l768", 1, 32, 32, 128, 768, 512, 32),
        # the same at 2048 positions
        _attend("attend_l2048", 1, 32, 32, 128, 2048, 1024, 32),
        # batch 32, 28 query heads on 4 kv heads
        _attend("attend_batch32", 32, 28, 4, 128, 1024, 512, 32),
        # the last position of a long sequence, one at a time
        _attend("attend_token_long", 1, 28, 4, 128, 131072, 131071, 1),
        # a block of long, padded sequences that sees its surroundings and the first positions
        _attend("attend_window", 8, 32, 8, 128, 16384, 8192, 32, lens="ragged", left=512,
                right=512, sinks=4),
        # odd sizes, one sequence without a visible position
        _attend("attend_window_odd", 3, 8, 2, 64, 1021, 500, 17, lens="ragged_empty", left=200,
                right=33, sinks=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST = {"bytes": 70e6, "flops": 14e9, "cache": 1 << 20}


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "attend", "attend"])
        d = rng.choice([64, 128, 128])
        b = _log(rng, 1, 64)
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
        L = _log(rng, 1, 131072)
        if op == "attend":
            block = min(L, _log(rng, 1, 128))
            start = rng.randint(0, L - block)
            windowed = rng.random() < 0.5
            case = _attend("", b, hkv * rng.choice([1, 1, 2, 4, 5, 7]), hkv, d, L, start, block,
                           rng.choice(["full", "ragged", "ragged_empty"]),
                           _log(rng, 1, 2048) - 1 if windowed else -1,
                           _log(rng, 1, 2048) - 1 if windowed and rng.random() < 0.8 else -1,
                           rng.randint(0, 64) if windowed else 0)
        else:
            n = _log(rng, 1, L)
            start = rng.randint(0, L - n)
            dtype = rng.choice(["bf16", "bf16", "f32"])
            if op == "write":
                case = _write("", b, hkv, d, L, start, n, dtype, rng.choice(["token", "head"]))
            else:
                case = _read("", b, hkv, d, L, start, n, dtype)
        del case["name"]
        w = work(case)
        if (op != "attend" or w["flops"]) and w["bytes"] <= MOST["bytes"] \
                and w["flops"] <= MOST["flops"] and b * hkv * L <= MOST["cache"]:
            return case


# ------------------------------------------------------------------ what a case is
def _lens(case):
    b, L = case["b"], case["L"]
    if case["lens"] == "full":
        return [L] * b
    lens = [max(1, L - (L * i * 5) // (9 * b)) for i in range(b)]
    if case["lens"] == "ragged_empty" and b > 1:
        lens[b // 2] = 0
        if b > 2:
            lens[0] = 1
    return lens


def _ranges(case, n):
    """The visible positions of a sequence with n valid ones: [0, a) and [lo, hi)."""
    lo = 0 if case["left"] < 0 else max(0, case["start"] - case["left"])
    hi = case["L"] if case["right"] < 0 else min(case["L"],
                                                 case["start"] + case["block"] + case["right"])
    first, hi = min(case["sinks"], n), min(hi, n)
    lo = min(lo, hi)
    return (first, lo, hi) if first < lo else (0, 0, max(first, hi))


def _visible(case):
    total = 0
    for n in _lens(case):
        a, lo, hi = _ranges(case, n)
        total += a + hi - lo
    return total


def work(case):
    d = case["d"]
    q4 = d // 2 + d // GROUP
    if case["op"] == "attend":
        rows = case["b"] * case["block"] * case["hq"]
        seen = _visible(case)
        return {"bytes": 2 * seen * case["hkv"] * q4 + rows * (2 * 2 * d + 4),
                "flops": 4 * case["block"] * case["hq"] * seen * d}
    rows = 2 * case["b"] * case["n"] * case["hkv"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "write":
        return {"bytes": rows * (d * e + q4 + d * 2), "flops": 0}
    return {"bytes": rows * (q4 + d * e), "flops": 0}


# --------------------------------------------------------------------- plain forms
def _quantise(x):
    """(codes, scales) of f32 rows x [..., d]: uint8 [..., d/2] and uint8 [..., d/16]."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    s8 = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.to(torch.float32).unsqueeze(-1)
    r = torch.where(s > 0, g / s, torch.zeros_like(g))
    a = r.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8)
            + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    code = torch.where(r < 0, code | 8, code).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8)


def _values(codes, scales):
    """f32 values of codes uint8 [..., d/2] under scales uint8 [..., d/16]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0,
                          -3.0, -4.0, -6.0], device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).to(torch.float32)
    return table[nib.to(torch.int32)] * s.repeat_interleave(GROUP, -1)


def _plain_write(st):
    c = st["case"]
    rows = slice(c["start"], c["start"] + c["n"])
    back = []
    for x, codes, scales in ((st["k_new"], st["k"], st["k_scale"]),
                             (st["v_new"], st["v"], st["v_scale"])):
        q, s = _quantise(x.transpose(1, 2).float())
        codes[:, :, rows] = q
        scales[:, :, rows] = s
        back.append(_values(codes[:, :, rows], scales[:, :, rows]).transpose(1, 2)
                    .to(torch.bfloat16).contiguous())
    return {"k": back[0], "v": back[1]}


def _plain_read(st):
    c = st["case"]
    rows = slice(c["start"], c["start"] + c["n"])
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    k, v = (_values(codes[:, :, rows], scales[:, :, rows]).transpose(1, 2).to(dt).contiguous()
            for codes, scales in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])))
    return {"k": k, "v": v}


def _plain_attend(st):
    c = st["case"]
    b, B, hq, d = st["q"].shape
    k, v = _values(st["k"], st["k_scale"]), _values(st["v"], st["v_scale"])
    grp = hq // c["hkv"]
    q = st["q"].float().reshape(b, B, c["hkv"], grp, d).permute(0, 2, 3, 1, 4)
    z = q.reshape(b, c["hkv"], grp * B, d) @ k.transpose(2, 3) * FDL_SCALE[d]
    j = torch.arange(c["L"], device=z.device)
    near = (j >= (c["start"] - c["left"] if c["left"] >= 0 else 0)) & \
        (j < (c["start"] + B + c["right"] if c["right"] >= 0 else c["L"]))
    seen = (near | (j < c["sinks"])) & (j < st["kv_len"].unsqueeze(1))          # [b, L]
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).reshape(b, hq, B)
    out = out.reshape(b, c["hkv"], grp, B, d).permute(0, 3, 1, 2, 4).reshape(b, B, hq, d)
    return {"out": out.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------------- the framework's calls
_ctx = None


def _context():
    global _ctx
    if _ctx is None:
        from block_kv_cache_b200 import fdllm
        _ctx = fdllm.Context(torch.cuda.current_device())
    return _ctx


def _run_own(st):
    from block_kv_cache_b200 import fdllm
    c, ctx = st["case"], _context()
    cache = fdllm.Kv4Cache(st["k"], st["k_scale"], st["v"], st["v_scale"])
    if c["op"] == "write":
        ctx.kv4_store(st["k_new"], st["v_new"], cache, c["start"])
        k, v = ctx.kv4_load(cache, c["start"], c["n"])
        return {"k": k, "v": v}
    if c["op"] == "read":
        k, v = ctx.kv4_load(cache, c["start"], c["n"],
                            dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        return {"k": k, "v": v}
    out, lse = ctx.kv4_attention(st["q"], cache, c["start"],
                                 kv_len=None if c["lens"] == "full" else st["kv_len"],
                                 window=(c["left"], c["right"]), sinks=c["sinks"], want_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return (_plain_write if op == "write" else _plain_read if op == "read" else
            _plain_attend)(state)


# ------------------------------------------------------------------------ inputs
def _rows(gen, shape, keys, dtype=torch.float32):
    """Fresh rows as a projection gives them: keys with a few large channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if keys:
        d = shape[-1]
        big = torch.rand(d, generator=gen, device="cuda")
        x = x * torch.where(big > 0.94, 6.0, 0.5 + big)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    b, hkv, d, L = case["b"], case["hkv"], case["d"], case["L"]
    st = {"case": dict(case)}
    for name in ("k", "v"):
        st[name], st[name + "_scale"] = _quantise(_rows(gen, (b, hkv, L, d), name == "k"))
    if case["op"] == "write":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        n = case["n"]
        for name in ("k", "v"):
            if case["order"] == "token":
                x = _rows(gen, (b, n, hkv, d), name == "k", dt)
            else:      # [b, n, Hkv, d] seen in a head-major buffer
                x = _rows(gen, (b, hkv, n, d), name == "k", dt).transpose(1, 2)
            st[name + "_new"] = x
    if case["op"] == "attend":
        st["q"] = _rows(gen, (b, case["block"], case["hq"], d), False, torch.bfloat16)
        st["kv_len"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    return st


# ----------------------------------------------------------------- 64-bit definition
def _round64(x, bits, low):
    """x rounded to `bits` fraction bits of its own power of two, at least 2^low, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** low))).clamp(min=low) - bits)
    return torch.round(x / step) * step


def _quantised64(x):
    """What rows x stand for after the cache, in float64."""
    g = x.double().unflatten(-1, (-1, GROUP))
    s = _round64(g.abs().amax(-1, keepdim=True) / 6, 3, -6).clamp(max=448)
    r = torch.where(s > 0, g / torch.where(s > 0, s, 1.0), 0.0)
    return (torch.sign(r) * _round64(r.abs(), 1, 0).clamp(max=6) * s).flatten(-2)


def _stored64(codes, scales):
    """What stored codes and scales stand for, in float64, from their bits."""
    c = torch.stack((codes.long() % 16, codes.long() // 16), -1).flatten(-2)
    e, m = c % 8 // 2, c % 2
    mag = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m.double() / 2), m.double() / 2)
    sc = scales.long()
    se, sm = sc % 128 // 8, sc % 8
    s = torch.where(se > 0, torch.exp2(se.double() - 7) * (1 + sm.double() / 8),
                    sm.double() * 2.0 ** -9)
    return torch.where(c >= 8, -mag, mag) * s.repeat_interleave(GROUP, -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return {"k": _quantised64(st["k_new"]).contiguous(),
                "v": _quantised64(st["v_new"]).contiguous()}
    rows = slice(case.get("start", 0), case.get("start", 0) + case.get("n", 0))
    if case["op"] == "read":
        return {n: _stored64(st[n][:, :, rows], st[n + "_scale"][:, :, rows])
                .transpose(1, 2).contiguous() for n in ("k", "v")}
    b, B, hq, d = st["q"].shape
    grp = hq // case["hkv"]
    out = torch.zeros((b, B, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq, B), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lens(case)):
        a, lo, hi = _ranges(case, n)
        keys = [j for j in (range(a), range(lo, hi)) if len(j)]
        if not keys:
            continue
        for h in range(case["hkv"]):
            k, v = (torch.cat([_stored64(st[x][i, h, j.start:j.stop],
                                         st[x + "_scale"][i, h, j.start:j.stop]) for j in keys])
                    for x in ("k", "v"))
            q = st["q"][i, :, h * grp:(h + 1) * grp].double()
            z = torch.einsum("igd,jd->gij", q, k) / math.sqrt(d)
            lse[i, h * grp:(h + 1) * grp] = torch.logsumexp(z, -1)
            out[i, :, h * grp:(h + 1) * grp] = torch.einsum("gij,jd->igd", torch.softmax(z, -1), v)
    return {"out": out, "lse": lse}
