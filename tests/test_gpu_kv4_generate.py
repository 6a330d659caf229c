"""fdl_generate with the layers' K/V held in 4 bits: the same steps and tokens as the decode
composed of the library's calls (each tested against the oracle on its own), for the DualCache
and the PrefixCache, with the host loop and the device loop; and its refusals."""
import numpy as np
import pytest
import torch

from block_kv_cache_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    from block_kv_cache_b200 import fdllm
    c = fdllm.Context(0)
    yield c
    c.close()


def _params(seed, hq, hkv, bias, layers=2):
    return synth.model_params(vocab=512, hidden=256, n_layers=layers, n_q_heads=hq,
                              n_kv_heads=hkv, head_dim=128, ffn=512, seed=seed, dtype="bf16",
                              qkv_bias=bias, w_std=0.06, lm_std=0.15)


def _rope(w, L):
    from block_kv_cache_b200 import fdllm
    s = w.shape
    return torch.from_numpy(fdllm.rope_table(s.rope_theta, L, 128)).cuda()


def composed(ctx, w, prompt, gen, B, tau, cache, bias=None):
    """The decode out of single calls: (x [b, L], steps)."""
    from block_kv_cache_b200 import fdllm
    s = w.shape
    b, P = prompt.shape
    L = P + gen
    D, F, hq, hkv = s.hidden, s.ffn, s.n_q_heads, s.n_kv_heads
    x = torch.full((b, L), s.mask_id, dtype=torch.int32, device="cuda")
    x[:, :P] = prompt
    masked = torch.zeros((b, L), dtype=torch.uint8, device="cuda")
    masked[:, P:] = 1
    caches = [fdllm.Kv4Cache.empty(b, hkv, L, 128) for _ in w.layers]
    rope = _rope(w, L)
    kf, vf = (torch.empty((b, hkv, L, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    seq = torch.arange(b, device="cuda", dtype=torch.int32)[:, None] * L

    def forward(first, n, full):
        """Hidden rows of positions [first, first + n) of every sequence, the K/V as the
        library holds them."""
        rows = b * n
        pos = torch.arange(first, first + n, device="cuda", dtype=torch.int32)
        h = ctx.embed(x, w.embed, row_map=(seq + pos).reshape(-1).contiguous())
        xb = torch.empty((rows, D), dtype=torch.bfloat16, device="cuda")
        q = torch.empty((b, n, hq, 128), dtype=torch.bfloat16, device="cuda")
        for Lw, c in zip(w.layers, caches):
            ctx.rmsnorm(h, Lw["attn_norm"], s.rms_eps, out=xb)
            ctx.qkv_rope_store(xb, Lw["w_qkv"], rope, q, kf, vf, n_q_heads=hq, rows_per_seq=n,
                               pos0=first, bias=Lw.get("bias"))
            if full:
                if first:
                    ctx.kv4_load(c, 0, first, k_out=kf[:, :, :first].transpose(1, 2),
                                 v_out=vf[:, :, :first].transpose(1, 2))
                o = ctx.full_attention(q, kf, vf, q_start=first)
                if not first:
                    ctx.kv4_store(kf.transpose(1, 2), vf.transpose(1, 2), c, 0)
            else:
                ctx.kv4_store(kf[:, :, first:first + n].transpose(1, 2),
                              vf[:, :, first:first + n].transpose(1, 2), c, first)
                o = ctx.kv4_attention(q, c, first)
            ctx.linear_residual(o.reshape(rows, hq * 128), Lw["wo"], h)
            ctx.ffn(xb, Lw["w_gu"], Lw["wd"], h, norm_w=Lw["ffn_norm"], eps=s.rms_eps)
        return h.reshape(b, n, D)

    steps = 0
    for st in range(P, L, B):
        first = True
        while True:
            if first:
                h = forward(0, L, True)[:, st:st + B]
            elif cache == "prefix":
                h = forward(st, L - st, True)[:, :B]
            else:
                h = forward(st, B, False)
            first = False
            xn = ctx.rmsnorm(h.reshape(b * B, D).contiguous(), w.final_norm, s.rms_eps)
            bt = bv = None
            if bias is not None:
                bt, bv = (t[:, st - P:st - P + B].reshape(-1).contiguous() for t in bias)
            conf, tok = ctx.lmhead_confidence(xn, w.lm_head, bt, bv)
            left = ctx.threshold_unmask(conf.reshape(b, B), tok.reshape(b, B), x, masked, st, tau)
            steps += 1
            if not left.any():
                break
    return x, steps


CASES = [(0, 0.9, 2, 2, False, 2, 64, 64, 32, "dual"), (1, 0.5, 4, 2, True, 3, 64, 64, 32, "dual"),
         (2, 1.0, 2, 1, False, 1, 32, 32, 32, "dual"), (3, 0.9, 8, 1, False, 2, 64, 64, 16, "dual"),
         (4, 0.9, 4, 2, True, 2, 64, 64, 32, "prefix"), (5, 0.9, 4, 4, False, 2, 32, 64, 32, "prefix"),
         (6, 0.9, 4, 4, False, 2, 64, 64, 64, "dual")]


def _bias(seed, mask_id, b, gen):
    g = synth.rng(seed + 60)
    return (torch.from_numpy(g.integers(0, mask_id, (b, gen)).astype(np.int32)).cuda(),
            torch.from_numpy(g.uniform(0.0, 16.0, (b, gen)).astype(np.float32)).cuda())


@pytest.mark.parametrize("seed,tau,hq,hkv,bias,b,Lp,gen,B,cache", CASES)
def test_generate_equals_its_calls(ctx, seed, tau, hq, hkv, bias, b, Lp, gen, B, cache):
    """At these shapes no projection splits K, so both runs are bit-identical."""
    from block_kv_cache_b200.model import DeviceWeights
    P = _params(seed, hq, hkv, bias)
    w = DeviceWeights.from_params(P)
    prompt = torch.from_numpy(synth.prompt_ids(seed, b, Lp, P.mask_id)).cuda()
    plant = _bias(seed, P.mask_id, b, gen)
    x_c, s_c = composed(ctx, w, prompt, gen, B, tau, cache, plant)
    m = w.native()
    for device_loop in (False, True, True):
        x, s = ctx.generate(m, prompt, gen, block=B, tau=tau, cache=cache, kv="4bit",
                            bias_tok=plant[0], bias_val=plant[1], device_loop=device_loop)
        ctx.device_status()
        assert s == s_c, device_loop
        assert torch.equal(x, x_c), device_loop
    assert (x[:, Lp:] != P.mask_id).all()


def test_formats_alternate_on_one_context(ctx):
    """A device-loop decode of one format does not launch the other's graph."""
    from block_kv_cache_b200.model import DeviceWeights
    P = _params(7, 4, 2, False)
    w = DeviceWeights.from_params(P)
    prompt = torch.from_numpy(synth.prompt_ids(7, 2, 64, P.mask_id)).cuda()
    m = w.native()
    want = {kv: ctx.generate(m, prompt, 64, block=32, tau=0.9, kv=kv) for kv in ("bf16", "4bit")}
    for kv in ("4bit", "bf16", "4bit"):
        x, s = ctx.generate(m, prompt, 64, block=32, tau=0.9, kv=kv, device_loop=True)
        assert s == want[kv][1] and torch.equal(x, want[kv][0]), kv


def test_split_projections_decode_every_position(ctx):
    """Shapes whose projections split K (and whose sums depend on the order of atomics): the
    prompt is kept, every position decoded, one per step at tau = 1."""
    from block_kv_cache_b200.model import DeviceWeights, ModelShape
    sh = ModelShape(4096, 1024, 2, 8, 2, 1024, 4095, 128, qkv_bias=True)
    w = DeviceWeights.random(sh, seed=5)
    prompt = torch.from_numpy(synth.prompt_ids(9, 3, 96, sh.mask_id)).cuda()
    x, steps = ctx.generate(w.native(), prompt, 64, block=32, tau=1.0, kv="4bit")
    ctx.device_status()
    assert steps == 64
    assert torch.equal(x[:, :96], prompt)
    assert (x >= 0).all() and (x < sh.vocab).all() and (x[:, 96:] != sh.mask_id).all()


def test_host_prompt_and_workspace(ctx):
    from block_kv_cache_b200 import fdllm
    from block_kv_cache_b200.model import DeviceWeights
    P = _params(8, 4, 2, False, layers=6)
    w = DeviceWeights.from_params(P)
    m = w.native()
    L = fdllm.load()
    size = {kv: L.fdl_generate_workspace_bytes_kv(ctx._h, m._h, 2, 2048, 32, kv) for kv in (0, 1)}
    assert size[0] == L.fdl_generate_workspace_bytes(ctx._h, m._h, 2, 2048, 32)
    bf16 = 2 * 2 * 2 * 2048 * 128 * 2                        # K and V of a layer
    scratch = ctx.kv4_attention_workspace_bytes(fdllm.Kv4AttnDesc(
        2, 4, 2, 128, 2048, 0, 32, fdllm.FDL_BF16, 0.0, -1, -1, 0))
    # 4.5 bits per value, one layer in bf16, and the attention's partial results
    saved = 6 * bf16 - (bf16 + 6 * bf16 * 9 // 32 + scratch)
    assert abs((size[0] - size[1]) - saved) <= 64 * 256
    assert L.fdl_generate_workspace_bytes_kv(ctx._h, m._h, 2, 2048, 32, 2) == 0
    prompt = torch.from_numpy(synth.prompt_ids(8, 2, 64, P.mask_id))
    x, _ = ctx.generate(m, prompt, 64, block=32, tau=0.9, kv="4bit")
    y, _ = ctx.generate(m, prompt.cuda(), 64, block=32, tau=0.9, kv="4bit")
    assert not x.is_cuda and torch.equal(x, y.cpu())


@pytest.mark.parametrize("bad", [dict(cache="none"), dict(batching="compact"),
                                 dict(batching="per_sequence")])
def test_refusals(ctx, bad):
    from block_kv_cache_b200 import fdllm
    from block_kv_cache_b200.model import DeviceWeights
    P = _params(9, 2, 2, False)
    m = DeviceWeights.from_params(P).native()
    prompt = torch.from_numpy(synth.prompt_ids(9, 2, 64, P.mask_id)).cuda()
    with pytest.raises(fdllm.FdlError) as e:
        ctx.generate(m, prompt, 64, block=32, kv="4bit", **bad)
    assert e.value.code == fdllm.FDL_EINVAL and "4-bit" in str(e.value)
