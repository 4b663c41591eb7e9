"""Plain 64-bit definitions of the serving operators (rotary positions, key/value cache,
decode of drafted tokens over it) on the CPU, for the parity tests."""
from __future__ import annotations

import math

import torch

MAX_CODE = {"e4m3": 448.0, "int8": 127.0}


def frequencies(dim, base=10000.0, scaling="none", factor=1.0, orig_len=4096, beta_fast=32.0, beta_slow=1.0,
                attn_factor=0.0):
    """(radians per position of each pair, factor of the rotated values)."""
    if scaling == "ntk":
        base = base * factor ** (dim / max(dim - 2, 1))
    out = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        if scaling == "linear":
            f /= factor
        if scaling == "by_parts":
            keep = min(1.0, max(0.0, (orig_len * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)))
            f = f * (1 - keep) / factor + f * keep
        out.append(f)
    g = attn_factor if attn_factor > 0 else (0.1 * math.log(factor) + 1 if scaling == "by_parts" else 1.0)
    return torch.tensor(out, dtype=torch.float64), g


def rotate(x, pos, dim, layout="half", inverse=False, **kw):
    """x [B, N, H, d] in float64 with its pairs rotated at pos [B, N], and for each element
    the sum of the magnitudes of the terms that it is made of."""
    f, g = frequencies(dim, **kw)
    ang = pos.double()[:, :, None, None] * f
    c, s = g * ang.cos(), g * ang.sin() * (-1 if inverse else 1)
    x = x.double()
    y, mag = x.clone(), x.abs().clone()
    ia = torch.arange(dim // 2) if layout == "half" else 2 * torch.arange(dim // 2)
    ib = ia + (dim // 2 if layout == "half" else 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = g * (a.abs() + b.abs())
    return y, mag


def dequantise(codes, scale):
    """codes [B, cap, H_kv, d] (bf16, e4m3 or int8) times scale [B, H_kv, cap], float64."""
    x = codes.cpu().double()
    return x if scale is None else x * scale.cpu().double().transpose(1, 2)[..., None]


def decode_tree(q, k, v, mask, lens, words, *, w, R, scale=None, vs=None):
    """q [B, T, H, d]; k, v [B, cap, H_kv, d] float64; mask [B, R, cap]; lens, words: lists.
    Returns float64 o [B, T, H, d], lse [B, H, T], and per output the magnitudes
    m = sum_j p_j |v_j| (as o), s = max_j sum_c |q_c k_jc| scale (as lse) and, with the
    scales vs [B, H_kv, cap] of an 8-bit cache, z = max_j (p_j vs_j) sum_j |code_j| (as o)."""
    B, T, H, d = q.shape
    H_kv = k.shape[2]
    scale = scale or 1 / math.sqrt(d)
    q = q.cpu().double()
    mask = mask.cpu().long() & 0xffffffff
    o, m = torch.zeros(B, T, H, d, dtype=torch.float64), torch.zeros(B, T, H, d, dtype=torch.float64)
    zz = torch.zeros(B, T, H, d, dtype=torch.float64)
    lse, s = torch.full((B, H, T), -math.inf, dtype=torch.float64), torch.zeros(B, H, T, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        bits = [int(x) & ((1 << T) - 1) for x in words[b]]
        depth = [bin(x).count("1") - 1 for x in bits]
        for t in range(T):
            if not bits[t]:
                continue
            for h in range(H):
                kvh = h // (H // H_kv)
                r = kvh // (H_kv // R)
                keys = []
                for j in range(n + T):
                    if j >= n and not bits[t] >> (j - n) & 1:
                        continue
                    pos = j if j < n else n + depth[j - n]
                    if n + depth[t] - pos < w or int(mask[b, r, n + t]) & int(mask[b, r, j]):
                        keys.append(j)
                if not keys:
                    continue
                kk, vv = k[b, keys, kvh], v[b, keys, kvh]
                z = (kk @ q[b, t, h]) * scale
                lse[b, h, t] = torch.logsumexp(z, 0)
                p = (z - lse[b, h, t]).exp()
                o[b, t, h] = p @ vv
                m[b, t, h] = p @ vv.abs()
                if vs is not None:
                    size = vs[b, kvh, keys].cpu().double()
                    code = vv.abs() / size.clamp(min=1e-300)[:, None]
                    zz[b, t, h] = (p * size).max() * code.sum(0)
                s[b, h, t] = (kk.abs() @ q[b, t, h].abs()).max() * scale
    return o, lse, m, s, zz


def random_tree(rng, T, reach=8):
    """Ancestor words of a random tree of T drafted tokens (token 0 is the root)."""
    words = []
    for t in range(T):
        words.append((words[rng.randrange(max(0, t - reach), t)] if t else 0) | 1 << t)
    return words


def signed(words):
    return [[x - (1 << 64) if x >> 63 else x for x in row] for row in words]
