"""Decode of a batch behind one prefix, against plain 64-bit softmax attention over the prefix's
and the sequence's own keys, through the public entry point.

Tolerances as for decode_tree (test_serving_gpu): the same products and roundings, with two
partial results joined in fp32, three more roundings of 2^-24 of what is joined, inside the 2^-18:
|err| <= (u(P) + 4 d 2^-22 s + 2^-18) m + u(bf16) |o| + 2^-28 z, |err LSE| <= 2 d 2^-22 s + 2^-18
max(1, |LSE|), with m = sum p |v|, s the logits' products' magnitudes and, in 8 bits, z = max(p vs)
sum |code|.
"""
import dataclasses
import math
import random

import pytest
import torch

import serving_ref as ref

focus = pytest.importorskip("learned_centroid_gated_gb300")

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def u(dtype):
    return torch.finfo(dtype).eps / 2


def randn(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def masks(seed, K, top_k, *shape):
    at = torch.rand(*shape, K, generator=torch.Generator().manual_seed(seed)).topk(top_k, dim=-1).indices
    bits = (1 << at).sum(-1)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


def filled(p, seed):
    """A cache of random rows, as cache_write makes them."""
    c = focus.KVCache.empty(p)
    k, v = (randn(p.B, p.cap, p.H_kv, p.d_head, seed=seed + i).cuda() for i in (0, 1))
    focus.cache_write(p, c, k, v, masks(seed + 2, p.K, p.top_k, p.B, p.R, p.cap).cuda(), torch.zeros(p.B, **I32))
    return c


def values(c):
    """k, v [B, cap, H_kv, d] in float64, and v's scales [B, H_kv, cap] or None."""
    out = []
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        out.append(x.double() if s is None else x.double() * s.double().transpose(1, 2)[..., None])
    return out[0], out[1], c.v_scale


def plain(p, q, prefix, P, c, lens, words):
    B, T, H, d = q.shape
    g = H // p.H_kv
    pk, pv, ps = values(prefix)
    ck, cv, cs = values(c)
    shape, rows = (B, T, H, d), (B, H, T)
    o, m, z = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(3))
    lse, s = torch.full(rows, -math.inf, dtype=torch.float64, device="cuda"), torch.zeros(rows, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b]
        bits = [x & ((1 << T) - 1) for x in words[b]]
        depth = torch.tensor([bin(x).count("1") - 1 for x in bits], device="cuda")
        pos = torch.cat([torch.arange(P + n, device="cuda"), P + n + depth])
        may = torch.zeros(T, P + n + T, dtype=torch.bool, device="cuda")
        may[:, :P + n] = torch.tensor([x != 0 for x in bits], device="cuda")[:, None]
        may[:, P + n:] = torch.tensor([[bool(x >> t & 1) for t in range(T)] for x in bits], device="cuda")
        near = (P + n + depth)[:, None] - pos < p.w
        for r in range(p.R):
            mk = torch.cat([prefix.mask[0, r, :P], c.mask[b, r, :n + T]])
            see = may & (near | ((mk[P + n:, None] & mk) != 0))
            for kvh in range(r * p.H_kv // p.R, (r + 1) * p.H_kv // p.R):
                k = torch.cat([pk[0, :P, kvh], ck[b, :n + T, kvh]])
                v = torch.cat([pv[0, :P, kvh], cv[b, :n + T, kvh]])
                for h in range(kvh * g, kvh * g + g):
                    x = q[b, :, h].double()
                    a = torch.where(see, (x @ k.T) * p.scale, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                    total = torch.logsumexp(a, -1, keepdim=True)
                    w = torch.where(total > -math.inf, (a - total).exp(), torch.zeros_like(a))
                    some = see.any(-1)
                    lse[b, h] = total[:, 0]
                    vz = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))
                    o[b, :, h], m[b, :, h] = w @ vz, w @ vz.abs()
                    s[b, h] = torch.where(see, x.abs() @ k.abs().T * p.scale, torch.zeros_like(a)).amax(-1)
                    if cs is not None:
                        size = torch.cat([ps[0, kvh, :P], cs[b, kvh, :n + T]]).double()
                        code = vz.abs() / size.clamp(min=1e-300)[:, None]
                        z[b, :, h] = (w * size).amax(-1, keepdim=True) * torch.stack([(code * see[t, :, None]).sum(0) for t in range(T)])
                    assert bool((lse[b, h][~some] == -math.inf).all())
    return o, lse, m, s, z


def check(p, q, prefix, P, c, lens, words, o, lse):
    want, want_lse, m, s, z = plain(p, q, prefix, P, c, lens, words)
    ds = p.d_head * 2.0 ** -22 * s
    up = u(torch.bfloat16 if p.format == "bf16" else torch.float16)
    bound = (up + 4 * ds.transpose(1, 2)[..., None] + 2.0 ** -18) * m + u(torch.bfloat16) * want.abs() + 2.0 ** -28 * z
    err = (o.double() - want).abs()
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert bool((o[empty.transpose(1, 2)] == 0).all())
    lerr = (lse.double() - want_lse).abs()[~empty]
    lbound = (2 * ds + 2.0 ** -18 * want_lse.abs().clamp(min=1))[~empty]
    print("max err / bound: o %.2f lse %.2f" % (float((err / bound.clamp(min=1e-30)).max()), float((lerr / lbound).max()) if len(lerr) else 0))
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-30)).max())
    assert bool((lerr <= lbound).all()), float((lerr / lbound).max())


def params(**kw):
    base = dict(B=2, cap=64, H=8, H_kv=2, d_head=128, R=1, K=4, top_k=1, w=16, format="bf16")
    base.update(kw)
    return focus.CacheParams(**base)


def make(fmt, B, T, P, length, seed=0, slack=3, kind="chain", **kw):
    """(p, q, prefix, its params, cache, lens, words) of ragged sequences; one of them empty."""
    r = random.Random(seed + 17)
    lens = [0 if b == 1 else r.randrange(0, length + 1) for b in range(B)]
    lens[0] = length
    p = params(B=B, cap=length + T + 2, format=fmt, **kw)
    pp = dataclasses.replace(p, B=1, cap=P + slack)
    words = [ref.random_tree(r, T) if kind == "tree" else [(2 << t) - 1 for t in range(T)] for _ in range(B)]
    if kind == "tree" and T > 2:
        for b in range(0, B, 3):
            for t in range(T - max(1, T // 4), T):
                words[b][t] = 0
    q = randn(B, T, p.H, p.d_head, seed=seed + 5).cuda()
    return p, q, filled(pp, seed + 10), pp, filled(p, seed + 20), lens, words


def call(p, q, prefix, P, c, lens, words=None, **kw):
    tree = None if words is None else torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda")
    return focus.decode_shared(p, q, prefix, P, c, torch.tensor(lens, **I32), tree, **kw)


CASES = {
    "one": dict(B=1, T=1, P=1, length=1),
    "two_short": dict(B=2, T=1, P=31, length=9),
    "rows_16": dict(B=4, T=1, P=700, length=40),
    "rows_20": dict(B=5, T=1, P=333, length=40, w=600, K=8, top_k=2, R=2),
    "small_layer": dict(B=4, T=1, P=2000, length=300, H=12, H_kv=12, d_head=64, top_k=2, w=256),
    "one_run": dict(B=64, T=1, P=1900, length=60, H=32, H_kv=8),
    "odd_runs": dict(B=70, T=1, P=2001, length=30, H=32, H_kv=8, R=8, K=8, top_k=2, w=100),
    "one_kv_head": dict(B=67, T=1, P=3000, length=20, H=16, H_kv=1, w=1, K=32, top_k=4),
    "three_per_head": dict(B=33, T=1, P=1500, length=20, H=24, H_kv=8, d_head=64),
    "mha": dict(B=130, T=1, P=1100, length=9, H=8, H_kv=8, d_head=64, K=1, top_k=1),
    "rows_64": dict(B=16, T=1, P=7000, length=50, H=32, H_kv=8, w=2000),
    "trees": dict(B=9, T=8, P=1000, length=90, kind="tree"),
    "trees_many_rows": dict(B=9, T=8, P=1700, length=90, H=32, H_kv=8, kind="tree", w=40, K=8, top_k=2),
    "chains_64": dict(B=3, T=64, P=200, length=70),
    # one group a token, a prefix long enough: tokens sorted by group
    "sorted_small": dict(B=33, T=1, P=6144, length=30, H=32, H_kv=8, w=20, K=3),
    "sorted_runs": dict(B=150, T=1, P=8200, length=9, H=16, H_kv=8, w=40, K=4),
    "sorted_trees": dict(B=9, T=8, P=6200, length=90, H=32, H_kv=8, kind="tree", w=300, K=3),
    "sorted_many_groups": dict(B=40, T=1, P=65540, length=5, H=16, H_kv=1, w=1, K=32, d_head=64),
    # beside them: a key, a row or a group too few, as they stand
    "not_sorted_keys": dict(B=33, T=1, P=6143, length=30, H=32, H_kv=8, w=20, K=3),
    "not_sorted_rows": dict(B=32, T=1, P=6200, length=30, H=32, H_kv=8, w=20, K=3),
    "not_sorted_groups": dict(B=40, T=1, P=4200, length=30, H=32, H_kv=8, w=20, K=2),
    "many": dict(B=1000, T=1, P=700, length=3, d_head=64, top_k=2),
    "sorted_many": dict(B=700, T=3, P=8192, length=4, d_head=64, H=4, H_kv=2, kind="tree"),
    "trees_many_rows_4": dict(B=37, T=5, P=600, length=40, H=32, H_kv=8, kind="tree", w=30, K=8, top_k=2),
    # sorted, with rows enough for a merge of four heads at a time
    "sorted_trees_rows_4": dict(B=20, T=8, P=6200, length=60, H=32, H_kv=8, kind="tree", w=300, K=3),
    "none_meet": dict(B=8, T=1, P=500, length=10, K=32, top_k=1, w=3),
}


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_the_definition(name, fmt):
    kw = CASES[name]
    p, q, prefix, _, c, lens, words = make(fmt, **kw)
    P = kw["P"]
    ws = torch.empty(focus.decode_shared_workspace_size(p, q.shape[1], P), dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)
    tree = words if kw.get("kind") == "tree" else None
    o, lse = call(p, q, prefix, P, c, lens, tree, ws=ws)
    assert focus.get_status(ws) == 0
    check(p, q, prefix, P, c, lens, words, o, lse)
    o2, lse2 = call(p, q, prefix, P, c, lens, words)         # the same bits, and a NULL tree is the chain
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("name", ["sorted_small", "sorted_runs", "sorted_trees", "sorted_trees_rows_4"])
def test_masks_of_other_numbers_of_groups(name, fmt):
    """top_k is what the work is planned by: masks of none, of several or of all groups are what is seen."""
    kw = CASES[name]
    p, q, prefix, _, c, lens, words = make(fmt, **kw)
    g = torch.Generator().manual_seed(9)
    for cache in (prefix, c):
        cache.mask.copy_(torch.randint(-2 ** 31, 2 ** 31, cache.mask.shape, generator=g).to(torch.int32))
        pick = torch.randint(0, 4, cache.mask.shape, generator=g).cuda()
        cache.mask[pick == 0] = 0
        cache.mask[pick == 1] = 1 << 30
        cache.mask[pick == 2] &= 0x11
    tree = words if kw.get("kind") == "tree" else None
    o, lse = call(p, q, prefix, kw["P"], c, lens, tree)
    check(p, q, prefix, kw["P"], c, lens, words, o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_no_prefix_is_decode_tree(fmt):
    p, q, prefix, _, c, lens, words = make(fmt, B=7, T=3, P=50, length=200)
    o, lse = call(p, q, prefix, 0, c, lens)
    want, want_lse = focus.decode_tree(p, q, c, torch.tensor(lens, **I32))
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_agrees_with_decode_tree_behind_a_copied_prefix():
    """The same batch with the prefix in front of each sequence's own cache."""
    P = 800
    p, q, prefix, _, c, lens, words = make("int8", B=6, T=4, P=P, length=100, kind="tree", w=90, K=8, top_k=2)
    whole = dataclasses.replace(p, cap=P + p.cap)
    w = focus.KVCache.empty(whole)
    for name in ("k", "v"):
        getattr(w, name)[:, :P] = getattr(prefix, name)[:, :P]
        getattr(w, name)[:, P:] = getattr(c, name)
    for name in ("k_scale", "v_scale", "mask"):
        getattr(w, name)[:, :, :P] = getattr(prefix, name)[:, :, :P]
        getattr(w, name)[:, :, P:] = getattr(c, name)
    o, lse = call(p, q, prefix, P, c, lens, words)
    tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda")
    want, want_lse = focus.decode_tree(whole, q, w, torch.tensor([n + P for n in lens], **I32), tree)
    assert (o.float() - want.float()).abs().max().item() <= 2.0 ** -7 * want.float().abs().max().item()
    both = want_lse > -math.inf
    assert torch.equal(both, lse > -math.inf) and (lse[both] - want_lse[both]).abs().max().item() <= 1e-4


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", ["rows_16", "rows_64", "one_run", "trees_many_rows", "trees_many_rows_4", "sorted_runs", "sorted_trees",
                                  "sorted_trees_rows_4"])
def test_what_a_row_must_not_see_shows_in_no_result(name, fmt):
    """NaN and infinities in slots behind the prefix, in slots behind the drafted tokens, and in
    prefix keys that only some tokens see."""
    kw = dict(CASES[name], K=CASES[name]["K"] if "sorted" in name else 8, top_k=1, w=20, slack=100)
    p, q, prefix, pp, c, lens, words = make(fmt, **kw)
    P, T = kw["P"], kw["T"]
    bad = [(1, math.nan), (P // 2, math.inf), (P // 2 + 1, math.nan), (P - 30, math.nan)]
    for j, _ in bad:                       # of group 0, which the first sequence is in and the second is not
        prefix.mask[:, :, j] = 1
    c.mask[0], c.mask[1] = 1, 2
    clean, clean_lse = call(p, q, prefix, P, c, lens, words)

    def spoil(cache, b, j, value):
        for x in (cache.k, cache.v):
            if fmt == "bf16":
                x[b, j] = value
        for x in (cache.k_scale, cache.v_scale):
            if fmt != "bf16":
                x[b, :, j] = value
    for j in range(P, P + 100):
        spoil(prefix, 0, j, math.nan)
    prefix.mask[:, :, P:] = -1
    for b in range(p.B):
        for j in range(lens[b] + T, p.cap):
            spoil(c, b, j, -math.inf)
    o, lse = call(p, q, prefix, P, c, lens, words)
    assert torch.equal(o, clean) and torch.equal(lse, clean_lse)
    for j, value in bad:
        spoil(prefix, 0, j, value)
    o, lse = call(p, q, prefix, P, c, lens, words)
    own = torch.zeros(p.B, p.R, T, dtype=torch.int32, device="cuda")
    for b in range(p.B):
        own[b] = c.mask[b, :, lens[b]:lens[b] + T]
    hit = torch.zeros(p.B, p.R, T, dtype=torch.bool, device="cuda")
    for j, _ in bad:
        near = torch.tensor([[P + lens[b] + bin(x & (1 << T) - 1).count("1") - 1 - j < p.w for x in words[b]] for b in range(p.B)],
                            device="cuda")
        hit |= ((own & prefix.mask[:, :, j:j + 1]) != 0) | near[:, None]
    hit &= torch.tensor([[x != 0 for x in w] for w in words], device="cuda")[:, None]
    assert 0 < int(hit.sum()) < hit.numel()
    heads = hit.repeat_interleave(p.H // p.R, 1)                       # [B, H, T]
    rows = heads.transpose(1, 2)
    assert bool(o[rows].isnan().any(-1).all()) and bool(lse[heads].isnan().all())
    assert bool(o[~rows].isfinite().all())
    err = (o[~rows].float() - clean[~rows].float()).abs().max().item()
    assert err <= 2.0 ** -7 * clean.float().abs().max().item()
    live = ~heads & (clean_lse > -math.inf)
    assert (lse[live] - clean_lse[live]).abs().max().item() <= 1e-4


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", ["sorted_runs", "sorted_trees", "sorted_trees_rows_4"])
def test_spoilt_keys_in_the_windows_of_some_of_a_run(name, fmt):
    """Keys of no group near the prefix's end: of the tokens of one group, which share their tiles, those with
    short sequences see them in their windows, and the others' rows are worked out again without them."""
    kw = dict(CASES[name], w=30)
    p, q, prefix, _, c, lens, words = make(fmt, **kw)
    P, T = kw["P"], kw["T"]
    bad = [(P - 29, math.inf), (P - 25, math.nan)]       # what sees the first sees the second
    for j, _ in bad:
        prefix.mask[:, :, j] = 0
    clean, clean_lse = call(p, q, prefix, P, c, lens, words)
    for j, value in bad:
        if fmt == "bf16":
            prefix.k[0, j], prefix.v[0, j] = value, value
        else:
            prefix.k_scale[0, :, j], prefix.v_scale[0, :, j] = value, value
    o, lse = call(p, q, prefix, P, c, lens, words)
    hit = torch.tensor([[x != 0 and any(P + n + bin(x & (1 << T) - 1).count("1") - 1 - j < p.w for j, _ in bad) for x in words[b]]
                        for b, n in enumerate(lens)], device="cuda")              # [B, T]
    live = torch.tensor([[x != 0 for x in w] for w in words], device="cuda")
    group = torch.stack([c.mask[b, 0, n:n + T] for b, n in enumerate(lens)])
    assert any(bool((hit & (group == g)).any() and (live & ~hit & (group == g)).any()) for g in (1, 2, 4, 8))
    assert bool(o[hit].isnan().all()) and bool(lse.transpose(1, 2)[hit].isnan().all())
    assert bool(o[~hit].isfinite().all())
    assert (o[~hit].float() - clean[~hit].float()).abs().max().item() <= 2.0 ** -7 * clean.float().abs().max().item()
    rows = (live & ~hit)[:, None].expand_as(lse)
    assert (lse[rows] - clean_lse[rows]).abs().max().item() <= 1e-4


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scales_far_apart(fmt):
    for name in ("rows_16", "one_run", "rows_64"):
        kw = CASES[name]
        p, q, prefix, _, c, lens, words = make(fmt, **kw)
        g = torch.Generator().manual_seed(3)
        for cache in (prefix, c):
            size = torch.exp2(torch.randint(-30, 30, cache.v_scale.shape, generator=g).float()).cuda()
            cache.v_scale.mul_(size)
        o, lse = call(p, q, prefix, kw["P"], c, lens)
        check(p, q, prefix, kw["P"], c, lens, words, o, lse)


@pytest.mark.parametrize("name", ["odd_runs", "sorted_runs"])
def test_lengths_outside_the_cache_are_reported(name):
    kw = CASES[name]
    p, q, prefix, _, c, lens, words = make("bf16", **kw)
    want, want_lse = call(p, q, prefix, kw["P"], c, lens)
    bad = list(lens)
    bad[3], bad[69], bad[30] = -1, p.cap, 2147483647
    status = torch.zeros(1, **I32)
    ws = torch.empty(focus.decode_shared_workspace_size(p, 1, kw["P"]), dtype=torch.uint8, device="cuda")
    o, lse = call(p, q, prefix, kw["P"], c, bad, ws=ws, status=status)
    assert focus.get_status(ws) == -6 and focus.get_status(status) == -6
    hit = torch.zeros(p.B, dtype=torch.bool)
    hit[[3, 30, 69]] = True
    assert bool((o.cpu()[hit] == 0).all()) and bool((lse.cpu()[hit] == -math.inf).all())
    assert (o.cpu()[~hit].float() - want.cpu()[~hit].float()).abs().max().item() <= 2.0 ** -5
    assert bool(lse.cpu()[~hit].isfinite().all())
    call(p, q, prefix, kw["P"], c, lens, ws=ws)
    assert focus.get_status(ws) == 0


@pytest.mark.parametrize("name", ["one_run", "sorted_runs"])
def test_graph_with_growing_sequences_and_streams(name):
    kw = CASES[name]
    p, q, prefix, _, c, lens, _ = make("e4m3", **kw)
    P = kw["P"]
    n = torch.tensor(lens, **I32)
    ws = [torch.empty(focus.decode_shared_workspace_size(p, 1, P), dtype=torch.uint8, device="cuda") for _ in range(2)]
    focus.decode_shared(p, q, prefix, P, c, n, ws=ws[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = focus.decode_shared(p, q, prefix, P, c, n, ws=ws[0])
    for cut in (0, 5, 60):
        n.copy_(torch.tensor([min(x, cut) for x in lens], **I32))
        graph.replay()
        want, want_lse = call(p, q, prefix, P, c, [min(x, cut) for x in lens])
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(6):
        got.append(focus.decode_shared(p, q, prefix, P, c, n, ws=ws[i % 2], stream=streams[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) and torch.equal(y, want_lse) for x, y in got)


def test_a_part_that_times_out_leaves_nan_and_a_usable_context():
    """The prefix's kernel or the own part's with one arrival kept back: its waits run out, and every row
    has a part in it and is NaN, whatever the other kernel left.  The next call is right."""
    p, q, prefix, _, c, lens, words = make("bf16", **CASES["rows_64"])
    want, want_lse = call(p, q, prefix, 7000, c, lens)
    for _ in range(2):
        assert focus.ERRORS[focus.selftest_timeout_shared()] == "FOCUS_ERR_TIMEOUT"
    o, lse = call(p, q, prefix, 7000, c, lens)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_prefix_behind_four_gigabytes():
    P, H_kv = 2300000, 8
    p = params(B=3, cap=8, H=32, H_kv=H_kv, w=300, K=32, top_k=1)
    pp = dataclasses.replace(p, B=1, cap=P)
    prefix, c = focus.KVCache.empty(pp), filled(p, 3)
    prefix.mask.fill_(1 << 20)
    c.mask.fill_(1 << 3)
    prefix.mask[0, 0, P - 900:P - 880] = 1 << 3
    for x, seed in ((prefix.k, 1), (prefix.v, 2)):
        x[0, P - 1000:] = randn(1000, H_kv, 128, seed=seed).cuda()
    q = randn(3, 1, 32, 128, seed=4).cuda()
    o, lse = call(p, q, prefix, P, c, [7, 0, 3])
    end = focus.KVCache(prefix.k[:, P - 1000:].contiguous(), prefix.v[:, P - 1000:].contiguous(), None, None,
                        prefix.mask[:, :, P - 1000:].contiguous())
    check(p, q, end, 1000, c, [7, 0, 3], [[1]] * 3, o, lse)


def test_refusals():
    p, q, prefix, pp, c, lens, _ = make("bf16", B=3, T=2, P=20, length=10)
    for P in (-1, prefix.k.shape[1] + 1):
        with pytest.raises(focus.FocusError):
            call(p, q, prefix, P, c, lens)
    other = focus.KVCache.empty(dataclasses.replace(pp, format="int8"))
    two = focus.KVCache.empty(dataclasses.replace(pp, B=2))
    heads = focus.KVCache.empty(dataclasses.replace(pp, H=4, H_kv=4))
    for bad in (other, two, heads, focus.KVCache(prefix.k, prefix.v, None, None, prefix.mask[:, :, :-1].contiguous()),
                focus.KVCache(prefix.k.cpu(), prefix.v, None, None, prefix.mask)):
        with pytest.raises(focus.FocusError):
            call(p, q, bad, 5, c, lens)
    with pytest.raises(focus.FocusError):
        call(p, q, prefix, 5, c, lens, out=q)
    with pytest.raises(focus.FocusError):
        call(p, q, prefix, 5, c, lens, ws=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(focus.FocusError):
        call(p, q[:, :1].expand(3, 65, 8, 128).contiguous(), prefix, 5, c, lens)
