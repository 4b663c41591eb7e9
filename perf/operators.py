"""The serving and long-context operators on one GPU: rotary positions of queries and keys
(and their backward pass), writing a key/value cache in bf16 or in 8 bits, reading it back,
and the centroid-gated attention of one or of many drafted tokens over such a cache.

`listed()` gives the cases by name, `draw(rng)` more of the same ranges, `prepare` what a
program holds before the call, and `run` one call: in plain torch operations, or through the
framework's entry points where `own` is true.  `exact` computes the same from the definitions
in 64 bits.
"""
import functools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOP = {"e4m3": 448.0, "int8": 127.0}          # the largest code of an 8-bit row
CODES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TINY = 2.0 ** -100                            # a row below this is held as zeros


# ------------------------------------------------------------------------------- cases --
def _rope(name, **kw):
    c = {"name": name, "op": "rope", "B": 1, "N": 1, "H": 32, "H_kv": 8, "d": 128, "dim": 128,
         "layout": "half", "scaling": "none", "factor": 1.0, "dtype": "bf16", "packed": False,
         "given": False, "offset": 0, "bwd": False}
    c.update(kw)
    return c


def _store(name, op, **kw):
    c = {"name": name, "op": op, "B": 1, "cap": 4096, "T": 1, "H_kv": 8, "d": 128, "R": 1, "K": 4,
         "top_k": 1, "format": "e4m3", "rope": True, "ragged": False}
    c.update(kw)
    return c


def _tree(name, **kw):
    c = {"name": name, "op": "tree", "B": 1, "len": 4096, "T": 1, "H": 32, "H_kv": 8, "d": 128, "R": 1,
         "K": 4, "top_k": 1, "w": 1024, "format": "bf16", "ragged": False, "pad": False, "chain": False}
    c.update(kw)
    return c


def listed():
    return [
        # one generated token of 16 sequences whose contexts were stretched eightfold: latency
        _rope("rope_step_16", B=16, scaling="by_parts", factor=8.0, given=True),
        # the 32K-token layer's queries and keys, cut out of a packed projection
        _rope("rope_32k_layer", N=32768, H_kv=32, packed=True),
        # a training step's gradients at 128K tokens, grouped queries, interleaved pairs
        _rope("rope_bwd_128k", N=131072, layout="interleaved", scaling="linear", factor=4.0, bwd=True),
        # the small layer in fp32 with half of each head rotated, an odd number of tokens
        _rope("rope_partial_f32", N=4095, H=12, H_kv=12, d=64, dim=32, scaling="ntk", factor=2.0, dtype="f32"),
        # 32 sequences each append a token
        _store("write_step_32", "write", B=32, T=1, ragged=True),
        # a 32K-token prompt enters the cache
        _store("write_prompt_32k", "write", cap=33000, T=32768, H_kv=32, K=4, top_k=2, R=1),
        # the 128K-token prefix of a conversation is read back for a further prompt
        _store("read_prefix_128k", "read", cap=131072, T=131072, R=8, K=8, top_k=2),
        # prompts of different lengths are written in 8-bit integers and read back
        _store("write_read_int8", "write_read", B=6, cap=8192, T=5001, format="int8", ragged=True),
        # the next token of four short sequences, the small layer
        _tree("step_short_4", B=4, len=1000, H=12, H_kv=12, d=64, K=4, top_k=2, w=256, ragged=True),
        # the next token of 32 sequences of up to 32K tokens
        _tree("step_e4m3_32", B=32, len=32768, K=8, top_k=2, R=8, format="e4m3", ragged=True),
        # a tree of 16 drafted tokens behind 128K tokens
        _tree("tree16_int8_128k", len=131072, T=16, R=8, K=8, top_k=2, format="int8"),
        # 64 drafted tokens behind a million
        _tree("tree64_bf16_1m", len=1000000, T=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8), (32, 32), (12, 12), (16, 1), (24, 8), (8, 2)]


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "read", "write_read", "tree", "tree", "tree"])
    H, H_kv = rng.choice(HEADS)
    d = 64 if H == 12 else rng.choice([128, 128, 64])
    K, top_k = rng.choice([(4, 1), (4, 2), (8, 2), (16, 3), (1, 1), (32, 4)])
    R = rng.choice([1, H_kv])
    if op == "rope":
        B = rng.choice([1, 1, 2, 7])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        c = _rope("", B=B, N=_log(rng, 1, 131072 * 40 // ((H + H_kv) * B * (2 if dtype == "f32" else 1))), H=H, H_kv=H_kv,
                  d=d, dim=rng.choice([d, d, d // 2, d - 2 * rng.randrange(1, d // 4)]), dtype=dtype,
                  layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                  factor=rng.choice([2.0, 4.0, 8.5]), packed=rng.random() < 0.4, given=rng.random() < 0.4,
                  offset=rng.choice([0, 1, _log(rng, 2, 1 << 20)]), bwd=rng.random() < 0.4)
        if c["scaling"] == "none":
            c["factor"] = 1.0
        if c["given"]:
            c["offset"] = 0
    elif op == "tree":
        B = rng.choice([1, 1, 2, 5, 16, 32])
        T = rng.choice([1, _log(rng, 2, 64)])
        fmt = rng.choice(["bf16", "e4m3", "int8"])
        longest = min(1000000, 1000000 * 8 // (B * H_kv), 64 * 32 * 1000000 // (B * H * T) // R)
        c = _tree("", B=B, len=_log(rng, 1, longest), T=T, H=H, H_kv=H_kv, d=d, R=R, K=K, top_k=top_k,
                  w=_log(rng, 1, 2048), format=fmt, ragged=B > 1 and rng.random() < 0.7,
                  pad=T > 3 and rng.random() < 0.3, chain=T > 1 and rng.random() < 0.3)
    else:
        B = rng.choice([1, 1, 4, 32])
        T = rng.choice([1, _log(rng, 1, 32768 * 32 // (B * H_kv)), _log(rng, 1, 32768 * 32 // (B * H_kv))])
        if op == "read":
            fmt = rng.choice(["e4m3", "int8", "bf16"])
        else:
            fmt = rng.choice(["e4m3", "e4m3", "bf16"]) if op == "write" else rng.choice(["int8", "e4m3"])
        c = _store("", op, B=B, cap=T + rng.randrange(0, 1 + min(1000, 4 * T + 8)), T=T, H_kv=H_kv, d=d, R=R, K=K,
                   top_k=top_k, format=fmt, rope=op != "read" and rng.random() < 0.7, ragged=rng.random() < 0.5)
    del c["name"]
    return c


def _lens(case):
    """Tokens in the cache of each sequence before the drafted ones; one sequence is empty where they differ."""
    B, n = case["B"], case["len"]
    if not case["ragged"]:
        return [n] * B
    return [0 if b == B - 1 and B > 2 else max(1, n * ((b * 7) % B + 1) // B) for b in range(B)]


def _counts(case):
    """(first slot, tokens) of each sequence of a write or a read."""
    B, T, cap = case["B"], case["T"], case["cap"]
    if not case["ragged"]:
        return [cap - T] * B, [T] * B
    count = [T if b == 0 or T == 1 else T * b // B for b in range(B)]
    return [(cap - n) * (b + 1) // (B + 1) for b, n in enumerate(count)], count


def _miss(K, k):
    return math.comb(K - k, k) / math.comb(K, k)


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["N"] * (case["H"] + case["H_kv"]) * d
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2.0 * n * size + (4.0 * case["B"] * case["N"] if case["given"] else 0),
                "flops": 3.0 * n * case["dim"] / d}
    code = 2 if case["format"] == "bf16" else 1
    row = d * code + (4 if code == 1 else 0)                      # one head's key or value with its scale
    if case["op"] != "tree":
        rows = 2.0 * sum(_counts(case)[1]) * case["H_kv"]
        n = rows * (2 * d + row)
        if case["op"] == "write_read":
            n *= 2
        if case["op"] == "read":
            n += 2.0 * (case["B"] * case["T"] - sum(_counts(case)[1])) * case["H_kv"] * 2 * d
        else:
            n += 8.0 * sum(_counts(case)[1]) * case["R"]
        return {"bytes": n, "flops": 4.0 * rows * d}
    T, w, H, H_kv = case["T"], case["w"], case["H"], case["H_kv"]
    miss = _miss(case["K"], case["top_k"])
    bytes_ = flops = 0.0
    for n in _lens(case):
        near, far = min(n, w), max(0, n - w)
        read = near + far * (1 - miss ** T) + T
        bytes_ += read * 2 * H_kv * row + 4.0 * case["R"] * (n + T) + 2 * T * H * d * 2 + 4 * T * H
        flops += 4.0 * d * H * T * (near + far * (1 - miss) + 1)
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------ inputs --
def _rand(g, *shape, dtype=torch.bfloat16):
    """N(0, 1), in the given type."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return out


def _groups(g, K, top_k, *shape):
    """Group bitmasks with top_k of K bits, every set as likely."""
    n = math.prod(shape)
    if top_k == K:
        return torch.full(shape, (1 << K) - 1, dtype=torch.int32, device="cuda")
    at = torch.rand(n, K, generator=g, device="cuda").topk(top_k, dim=1).indices
    return (1 << at).sum(1).to(torch.int32).view(shape)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _fill(g, case, cap):
    """A cache that holds tokens in every slot: codes, scales and group masks."""
    B, H_kv, d, fmt = case["B"], case["H_kv"], case["d"], case["format"]
    c = {"mask": _groups(g, case["K"], case["top_k"], B, case["R"], cap), "k_scale": None, "v_scale": None}
    for x in "kv":
        if fmt == "bf16":
            c[x] = _rand(g, B, cap, H_kv, d)
        elif fmt == "int8":
            c[x] = torch.randint(-127, 128, (B, cap, H_kv, d), generator=g, device="cuda", dtype=torch.int8)
        else:
            c[x] = torch.empty(B, cap, H_kv, d, dtype=torch.float8_e4m3fn, device="cuda")
            flat = c[x].view(-1)
            for at in range(0, flat.numel(), 1 << 28):
                part = flat[at:at + (1 << 28)]
                part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(140.0).clamp_(-448.0, 448.0))
        if fmt != "bf16":
            c[x + "_scale"] = (torch.rand(B, H_kv, cap, generator=g, device="cuda") + 0.5) / (70.0 if fmt == "int8" else 140.0)
    return c


def _draft(seed, case):
    """Ancestors of each drafted token (itself among them) as bits, a row of no bits where there is no token."""
    import random
    r, rows = random.Random(seed), []
    for b in range(case["B"]):
        bits, n = [], case["T"]
        if case["pad"] and b % 2 == 0:
            n -= max(1, n // 4)
        for t in range(case["T"]):
            up = 0 if t == 0 or t >= n else bits[t - 1] if case["chain"] else bits[r.randrange(max(0, t - 8), t)]
            bits.append(0 if t >= n else up | 1 << t)
        rows.append([x - (1 << 64) if x >> 63 else x for x in bits])
    return rows


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 12345)
    B, d, H_kv = case["B"], case["d"], case["H_kv"]
    s = {"case": case}
    if case["op"] == "rope":
        N, H, dtype = case["N"], case["H"], DTYPES[case["dtype"]]
        if case["packed"]:
            both = _rand(g, B, N, H + 2 * H_kv, d, dtype=dtype)
            s["q"], s["k"] = both[:, :, :H], both[:, :, H:H + H_kv]
        else:
            s["q"], s["k"] = _rand(g, B, N, H, d, dtype=dtype), _rand(g, B, N, H_kv, d, dtype=dtype)
        s["positions"] = (torch.randint(0, 1 << 20, (B, N), generator=g, device="cuda", dtype=torch.int32)
                          if case["given"] else None)
        return s
    if case["op"] == "tree":
        lens = _lens(case)
        s["lens"], s["longest"] = _ints(lens), max(lens)
        s["cache"] = _fill(g, case, max(lens) + case["T"])
        s["q"] = _rand(g, B, case["T"], case["H"], d)
        s["tree"] = None if case["chain"] and not case["pad"] else _ints(_draft(seed, case), torch.int64)
        return s
    start, count = _counts(case)
    s["start"], s["count"] = _ints(start), _ints(count)
    s["cache"] = _fill(g, case, case["cap"])
    if case["op"] != "read":
        s["k"], s["v"] = _rand(g, B, case["T"], H_kv, d), _rand(g, B, case["T"], H_kv, d)
        s["mask"] = _groups(g, case["K"], case["top_k"], B, case["R"], case["T"])
    return s


# -------------------------------------------------------------------------- plain forms --
def _frequencies(dim, scaling, factor):
    """Radians per position of each pair, in 64 bits, and the factor of the rotated values."""
    base, grow = 10000.0, 1.0
    if scaling == "ntk":
        base *= factor ** (dim / max(dim - 2, 1))
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f / factor * (1 - keep) + f * keep
        grow = 0.1 * math.log(factor) + 1.0
    return f, grow


def _turn(x, angle, dim, layout, grow, back):
    """x rotated pair by pair by `angle` [.., .., 1, dim / 2] (64 bits), in fp32."""
    c, s = (grow * angle.cos()).float(), (grow * angle.sin()).float()
    if back:
        s = -s
    x = x.float()
    part, rest = x[..., :dim], x[..., dim:]
    if layout == "half":
        a, b = part[..., :dim // 2], part[..., dim // 2:]
        part = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([part, rest], -1) if dim < x.shape[-1] else part


def _plain_rope(s):
    c = s["case"]
    pos = s["positions"] if c["given"] else torch.arange(c["N"], device="cuda")[None] + c["offset"]
    f, grow = _frequencies(c["dim"], c["scaling"], c["factor"])
    angle = pos.double()[:, :, None, None] * f
    return [_turn(s[x], angle, c["dim"], c["layout"], grow, c["bwd"]).to(s[x].dtype) for x in "qk"]


def _plain_write(s):
    c, cache = s["case"], s["cache"]
    t = torch.arange(c["T"], device="cuda")[None]
    slot = s["start"][:, None].long() + t
    b, t = torch.nonzero(t < s["count"][:, None], as_tuple=True)
    at = slot[b, t]
    for x in "kv":
        rows = s[x][b, t].float()                                     # [n, H_kv, d]
        if x == "k" and c["rope"]:
            f, grow = _frequencies(c["d"], "none", 1.0)
            rows = _turn(rows, at.double()[:, None, None] * f, c["d"], "half", grow, False)
        if c["format"] == "bf16":
            cache[x][b, at] = rows.to(torch.bfloat16)
            continue
        top = rows.abs().amax(-1)
        some = top >= TINY
        codes = rows * torch.where(some, TOP[c["format"]] / top, 0.0)[..., None]
        codes = codes.round() if c["format"] == "int8" else codes
        cache[x].view(torch.uint8)[b, at] = codes.to(CODES[c["format"]]).view(torch.uint8)
        cache[x + "_scale"][b, :, at] = torch.where(some, top / TOP[c["format"]], 0.0)
    cache["mask"][b, :, at] = s["mask"][b, :, t]


def _plain_read(s):
    c, cache = s["case"], s["cache"]
    t = torch.arange(c["T"], device="cuda")[None]
    valid = t < s["count"][:, None]
    slot = torch.where(valid, s["start"][:, None].long() + t, 0)      # [B, T]
    b = torch.arange(c["B"], device="cuda")[:, None]
    out = []
    for x in "kv":
        rows = cache[x].view(torch.uint8 if c["format"] != "bf16" else torch.bfloat16)[b, slot].view(CODES[c["format"]]).float()
        if c["format"] != "bf16":
            rows = rows * cache[x + "_scale"].transpose(1, 2)[b, slot][..., None]
        out.append((rows * valid[:, :, None, None]).to(torch.bfloat16))
    return out


def _plain_tree(s):
    c, cache = s["case"], s["cache"]
    B, T, H, H_kv, R, d = c["B"], c["T"], c["H"], c["H_kv"], c["R"], c["d"]
    cap = cache["k"].shape[1]
    t, n = torch.arange(T, device="cuda"), torch.arange(cap, device="cuda")
    lens = s["lens"].long()
    bits = s["tree"] if s["tree"] is not None else ((2 << t) - 1).expand(B, T)
    up = (bits[:, :, None] >> t & 1).bool()                           # [B, T, T]
    depth = up.sum(-1) - 1                                            # [B, T]
    live = bits != 0
    u = (n - lens[:, None])                                           # [B, cap]: drafted token of a slot
    drafted, u = (u >= 0) & (u < T), u.clamp(0, T - 1)
    pos_q = lens[:, None] + depth                                     # [B, T]
    pos_k = torch.where(n < lens[:, None], n, lens[:, None] + depth.gather(1, u))
    see = live[:, :, None] & ((n < lens[:, None])[:, None] | drafted[:, None] & up.gather(2, u[:, None].expand(B, T, cap)))
    mask_q = cache["mask"].gather(2, (lens[:, None] + t)[:, None].expand(B, R, T))
    meet = (mask_q[..., None] & cache["mask"][:, :, None]) != 0       # [B, R, T, cap]
    see = see[:, None] & (meet | (pos_q[:, :, None] - pos_k[:, None] < c["w"])[:, None])
    x = {}
    for y in "kv":
        x[y] = cache[y].float()
        if c["format"] != "bf16":
            x[y] = x[y] * cache[y + "_scale"].transpose(1, 2)[..., None]
    q = s["q"].float().view(B, T, H_kv, H // H_kv, d).permute(0, 2, 3, 1, 4).reshape(B, H_kv, -1, d)
    p = (q @ x["k"].permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))      # [B, H_kv, gq T, cap]
    p.view(B, R, H // R, T, cap).masked_fill_(~see[:, :, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    some = top > -math.inf
    p.sub_(torch.where(some, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True, dtype=torch.float64)
    o = (p @ x["v"].transpose(1, 2)) / torch.where(some, total, 1.0).float()
    lse = (top.double() + torch.where(some, total, 1.0).log()).float()
    o = o.view(B, H_kv, H // H_kv, T, d).permute(0, 3, 1, 2, 4).reshape(B, T, H, d)
    return [o.to(torch.bfloat16), lse.view(B, H, T)]


def _stored(s):
    return {x: v for x, v in s["cache"].items() if v is not None}


# --------------------------------------------------------------------------- own calls --
@functools.lru_cache(maxsize=None)
def _plan(dim, layout, scaling, factor):
    import learned_centroid_gated_gb300 as focus
    return focus.Rope(dim=dim, layout=layout, scaling=scaling, factor=factor, orig_len=4096)


@functools.lru_cache(maxsize=None)
def _sizes(B, cap, H, H_kv, d, R, K, top_k, w, fmt):
    import learned_centroid_gated_gb300 as focus
    return focus.CacheParams(B=B, cap=cap, H=H, H_kv=H_kv, d_head=d, R=R, K=K, top_k=top_k, w=w, format=fmt)


def _own(s):
    import learned_centroid_gated_gb300 as focus
    c = s["case"]
    if c["op"] == "rope":
        call = focus.rope_bwd if c["bwd"] else focus.rope
        return list(call(_plan(c["dim"], c["layout"], c["scaling"], c["factor"]), s["q"], s["k"],
                         positions=s["positions"], offset=c["offset"]))
    k = s["cache"]
    cache = focus.KVCache(k["k"], k["v"], k["k_scale"], k["v_scale"], k["mask"])
    if c["op"] == "tree":
        p = _sizes(c["B"], k["k"].shape[1], c["H"], c["H_kv"], c["d"], c["R"], c["K"], c["top_k"], c["w"], c["format"])
        return list(focus.decode_tree(p, s["q"], cache, s["lens"], s["tree"]))
    p = _sizes(c["B"], c["cap"], c["H_kv"], c["H_kv"], c["d"], c["R"], c["K"], c["top_k"], 1, c["format"])
    if c["op"] != "read":
        rope = _plan(c["d"], "half", "none", 1.0) if c["rope"] else None
        focus.cache_write(p, cache, s["k"], s["v"], s["mask"], s["start"], s["count"], rope=rope)
        if c["op"] == "write":
            return _stored(s)
    return list(focus.cache_read(p, cache, c["T"], s["start"], s["count"]))


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "tree":
        return _plain_tree(state)
    if op != "read":
        _plain_write(state)
        if op == "write":
            return _stored(state)
    return _plain_read(state)


# ------------------------------------------------------------------- 64-bit definitions --
def _spin(x, pos, dim, layout, scaling, factor, back):
    """x in 64 bits with its pairs as complex numbers times factor * exp(i pos f); pos [..., 1]."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=x.device)
    base = 1e4 * factor ** (dim / max(dim - 2, 1)) if scaling == "ntk" else 1e4
    f = torch.exp(-2.0 * i / dim * math.log(base))
    size = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        ramp = ((4096 * f / math.tau - 1) / 31).clamp(0, 1)
        f, size = f * (ramp + (1 - ramp) / factor), 1 + math.log(factor) / 10
    turn = torch.polar(torch.full_like(pos * f, size), (-1.0 if back else 1.0) * pos * f)
    out = x.double().clone()
    if layout == "half":
        z = torch.complex(out[..., :dim // 2], out[..., dim // 2:dim]) * turn
        out[..., :dim // 2], out[..., dim // 2:dim] = z.real, z.imag
    else:
        z = torch.complex(out[..., 0:dim:2], out[..., 1:dim:2]) * turn
        out[..., 0:dim:2], out[..., 1:dim:2] = z.real, z.imag
    return out


def _e4m3(x):
    """The nearest number of 3 mantissa bits and exponents from -6, even ones in ties, in 64 bits."""
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
    return ((x / step).round() * step).clamp(-448, 448)


def _host(v):
    return {x: _host(y) for x, y in v.items()} if isinstance(v, dict) else [_host(y) for y in v] if isinstance(v, list) else v.cpu()


def exact(case, seed):
    s = prepare(case, seed)
    B, d = case["B"], case["d"]
    if case["op"] == "rope":
        pos = s["positions"] if case["given"] else (torch.arange(case["N"], device="cuda") + case["offset"]).expand(B, -1)
        return [_spin(s[x], pos.double()[:, :, None, None], case["dim"], case["layout"], case["scaling"],
                      case["factor"], case["bwd"]).cpu() for x in "qk"]
    cache, fmt = s["cache"], case["format"]
    held = {x: cache[x].double() for x in "kv"}
    scale = {x: None if fmt == "bf16" else cache[x + "_scale"].double() for x in "kv"}
    if case["op"] == "tree":
        return _exact_tree(s, held, scale)
    start, count = _counts(case)
    mask = cache["mask"]
    if case["op"] != "read":
        for b in range(B):
            at = slice(start[b], start[b] + count[b])
            mask[b, :, at] = s["mask"][b, :, :count[b]]
            for x in "kv":
                new = s[x][b, :count[b]].double()
                if x == "k" and case["rope"]:
                    new = _spin(new, torch.arange(start[b], start[b] + count[b], device="cuda").double()[:, None, None],
                                d, "half", "none", 1.0, False)
                if fmt != "bf16":
                    unit = new.abs().amax(-1) / TOP[fmt]
                    new = new / unit[..., None].clamp(min=1e-300)
                    new = _e4m3(new) if fmt == "e4m3" else new.round()
                    scale[x][b, :, at] = unit.T
                held[x][b, at] = new
    if case["op"] == "write":
        out = {"k": held["k"], "v": held["v"], "mask": mask}
        if fmt != "bf16":
            out |= {"k_scale": scale["k"], "v_scale": scale["v"]}
        return _host(out)
    out = []
    for x in "kv":
        got = torch.zeros(B, case["T"], case["H_kv"], d, dtype=torch.float64, device="cuda")
        for b in range(B):
            at = slice(start[b], start[b] + count[b])
            got[b, :count[b]] = held[x][b, at] if fmt == "bf16" else held[x][b, at] * scale[x][b, :, at].T[..., None]
        out.append(got)
    return _host(out)


def _exact_tree(s, held, scale):
    """Row by row: the keys that a drafted token may see, gathered, and their softmax."""
    c = s["case"]
    B, T, H, R, d = c["B"], c["T"], c["H"], c["R"], c["d"]
    per, heads = c["H_kv"] // R, H // R                                # key and query heads of a routing head
    if c["len"] * T * B > 1 << 27:
        return None
    o = torch.zeros(B, T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    draft = s["tree"].tolist() if s["tree"] is not None else [[(2 << t) - 1 for t in range(T)]] * B
    for b, n in enumerate(_lens(c)):
        place = torch.arange(n + T, device="cuda")
        depth = [bin(x & (2 ** 64 - 1)).count("1") - 1 for x in draft[b]]
        place[n:] = n + torch.tensor(depth, device="cuda")
        for t in range(T):
            bits = draft[b][t]
            if bits == 0:
                continue
            may = torch.ones(n + T, dtype=torch.bool, device="cuda")
            may[n:] = torch.tensor([bool(bits >> u & 1) for u in range(T)], device="cuda")
            close = place > n + depth[t] - c["w"]
            for r in range(R):
                m = s["cache"]["mask"][b, r, :n + T]
                keys = torch.nonzero(may & (close | (m & m[n + t]).bool())).flatten()
                q = s["q"][b, t, r * heads:(r + 1) * heads].double().view(per, heads // per, d)
                kv = {}
                for x in "kv":
                    kv[x] = held[x][b, keys, r * per:(r + 1) * per].transpose(0, 1)      # [per, n, d]
                    if scale[x] is not None:
                        kv[x] = kv[x] * scale[x][b, r * per:(r + 1) * per][:, keys, None]
                z = torch.baddbmm(torch.zeros((), dtype=torch.float64, device="cuda"), q, kv["k"].transpose(1, 2),
                                  alpha=d ** -0.5)
                total = torch.logsumexp(z, -1, keepdim=True)
                lse[b, r * heads:(r + 1) * heads, t] = total.flatten()
                o[b, t, r * heads:(r + 1) * heads] = ((z - total).exp() @ kv["v"]).reshape(heads, d)
    return _host([o, lse])
