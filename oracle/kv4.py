"""Float64 oracle of the 4-bit K/V cache: quantisation, the values a cache stands for, and the
block attention over its visible positions. numpy only; every rounding is the definition's.

Groups of 16 along the last dimension share scale = e4m3(max |x| / 6) (to nearest even, at most
448); code = e2m1(x / scale) (to nearest even, at most 6; 0 where x is 0 or the scale 0 or NaN, -0
where x < 0 rounds to 0).
"""
from __future__ import annotations

import numpy as np

GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                 for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def _nearest_even(x, grid):
    """Index of the entry of the ascending `grid` nearest to x >= 0, the even index on ties."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def kv4_quantise(x):
    """(codes, scales) uint8 [..., d/2] and [..., d/16] of rows x [..., d]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(g).max(-1)                                    # NaN if any is
        scale = np.where(np.isnan(amax), 127,
                         _nearest_even(np.minimum(np.nan_to_num(amax, posinf=1e300) / 6, 448.0),
                                       E4M3[:127])).astype(np.uint8)
        s = E4M3[scale][..., None]
        r = np.where(s > 0, np.abs(g) / np.where(s > 0, s, 1.0), 0.0)
        code = _nearest_even(np.minimum(np.nan_to_num(r, posinf=1e300), 6.0), E2M1)
    code = (code | np.where((g < 0) & (s > 0), 8, 0)).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def kv4_values(codes, scales):
    """Float64 values that codes under scales stand for."""
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    mag = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    sign = np.where(scales & 128, -1.0, 1.0)
    return mag * np.repeat(sign * E4M3[scales & 127], GROUP, -1)


def kv4_visible(seq_len, block_start, block_len, kv_len=None, window=(-1, -1), sinks=0):
    """Boolean [L]: the positions a block sees in a sequence of kv_len valid ones."""
    j = np.arange(seq_len)
    lo = -1 if window[0] < 0 else block_start - window[0]
    hi = seq_len if window[1] < 0 else block_start + block_len + window[1]
    return (j < (seq_len if kv_len is None else kv_len)) & ((j < sinks) | ((j >= lo) & (j < hi)))


def kv4_attention(q, k, v, seen, scale=None):
    """Attention of one sequence's block: q [B, Hq, d], k, v [Hkv, L, d], seen [L] ->
    (out [B, Hq, d], lse [Hq, B], spread [B, Hq, d]); spread = sum_j p_j |v_j|, the size that
    rounding errors of the probabilities are relative to."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    B, hq, d = q.shape
    grp = hq // k.shape[0]
    scale = d ** -0.5 if scale is None else scale
    out, spread = np.zeros((B, hq, d)), np.zeros((B, hq, d))
    lse = np.full((hq, B), -np.inf)
    if not seen.any():
        return out, lse, spread
    for h in range(hq):
        kk, vv = k[h // grp][seen], v[h // grp][seen]
        z = q[:, h] @ kk.T * scale
        m = z.max(1, keepdims=True)
        p = np.exp(z - m)
        l = p.sum(1, keepdims=True)
        out[:, h] = p @ vv / l
        spread[:, h] = p @ np.abs(vv) / l
        lse[h] = (m + np.log(l))[:, 0]
    return out, lse, spread
