"""Rotary positions, the key/value cache and the decode of drafted tokens over it, against
plain 64-bit definitions (serving_ref), through the public entry points.

Tolerances.  u(t) = eps(t) / 2 is the largest relative error of one rounding to type t.
* Rotation: cosine and sine are within 2^-22 (their own error of a few fp32 steps and the
  angle's 2^-24 half turns), each product and the sum round once in fp32, the result once in
  t: |err| <= u(t) |y| + 2^-20 (|a| + |b|) g, plus the type's smallest step.
* 8-bit codes: half a step of the row's scale (int8), or 2^-4 of the value with half of the
  smallest step 2^-10 below (e4m3); the scale has two fp32 roundings.
* Attention: the logits are fp32 sums of d exact products, off by at most d 2^-22 of the
  products' magnitudes s; P is rounded to bf16 (or, with 8-bit codes, to fp16) for the second
  product, the result to bf16: |err| <= (u(P) + 4 d 2^-22 s + 2^-18) m + u(bf16) |o| with
  m = sum p |v|, and |err LSE| <= 2 d 2^-22 s + 2^-18 max(1, |LSE|).  With 8-bit codes c and
  scales vs, fp16 holds p vs: the largest of a row is kept at 2^3 or more there (2^7 when the
  reference is set, up to 2^4 below it where a tile's scales differ by less than that), and
  below 2^-14 a rounding is off by up to 2^-25 absolute, that is 2^-28 of the largest:
  another 2^-28 max(p vs) sum |c|, which matters where the large rows' codes are 0.
"""
import dataclasses
import math
import random

import pytest
import torch

import serving_ref as ref

focus = pytest.importorskip("learned_centroid_gated_gb300")

pytestmark = pytest.mark.gpu


def u(dtype):
    return torch.finfo(dtype).eps / 2


def randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def random_masks(seed, K, top_k, *shape):
    g = torch.Generator().manual_seed(seed)
    at = torch.rand(*shape, K, generator=g).topk(top_k, dim=-1).indices
    bits = (1 << at).sum(-1)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


# --------------------------------------------------------------------------- rotation --
def close_rotation(y, want, mag, dtype):
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    bound = u(dtype) * want.abs() + 2.0 ** -20 * mag + tiny
    err = (y.cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


ROPES = [
    dict(dim=128, d=128), dict(dim=64, d=64), dict(dim=128, d=128, layout="interleaved"),
    dict(dim=64, d=128), dict(dim=32, d=64, layout="interleaved"), dict(dim=2, d=64), dict(dim=2, d=128, layout="interleaved"),
    dict(dim=54, d=128), dict(dim=52, d=64), dict(dim=126, d=128), dict(dim=102, d=128, layout="interleaved"),
    dict(dim=128, d=128, scaling="linear", factor=4.0), dict(dim=64, d=64, scaling="ntk", factor=8.5),
    dict(dim=128, d=128, scaling="by_parts", factor=16.0), dict(dim=4, d=64, scaling="ntk", factor=2.0),
    dict(dim=2, d=64, scaling="ntk", factor=2.0),
    dict(dim=96, d=128, scaling="by_parts", factor=3.0, orig_len=777, beta_fast=20.0, beta_slow=0.0, attn_factor=0.7),
    dict(dim=128, d=128, base=1e6),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("case", range(len(ROPES)))
@pytest.mark.parametrize("inverse", [False, True])
def test_rotation_matches_the_definition(dtype, case, inverse):
    kw = dict(ROPES[case])
    d, dim, layout = kw.pop("d"), kw.pop("dim"), kw.pop("layout", "half")
    B, N, H, H_kv = [(1, 1, 1, 1), (2, 7, 5, 1), (1, 33, 12, 12), (3, 5, 8, 2)][case % 4]
    plan = focus.Rope(dim=dim, layout=layout, **kw)
    q, k = randn(B, N, H, d, seed=case, dtype=dtype), randn(B, N, H_kv, d, seed=case + 50, dtype=dtype)
    call = focus.rope_bwd if inverse else focus.rope
    g = torch.Generator().manual_seed(case)
    for given in (False, True):
        offset = 0 if given else [0, 3, 1 << 20, 1 << 28][case % 4]
        pos = (torch.randint(-(1 << 28), 1 << 28, (B, N), generator=g) if given
               else torch.arange(N).expand(B, N) + offset)
        out = call(plan, q.cuda(), k.cuda(), offset=offset,
                   positions=pos.to(torch.int32).cuda() if given else None)
        for x, y in zip((q, k), out):
            want, mag = ref.rotate(x, pos, dim, layout, inverse, **kw)
            # (both sides' f and its product with pos are off by 2^-52 each: 2^-22 at 2^28)
            close_rotation(y, want, mag, dtype)
            assert torch.equal(y[..., dim:].cpu(), x[..., dim:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout,dim", [("half", 128), ("interleaved", 128), ("half", 50)])
def test_rotation_of_strided_views_in_place_and_alone(dtype, layout, dim):
    """Queries and keys cut out of a packed projection, outputs in place and into views,
    rows that start at odd elements, and queries without keys: the same bits as dense calls."""
    plan = focus.Rope(dim=dim, layout=layout)
    packed = randn(2, 9, 14, 128, seed=1, dtype=dtype).cuda()
    q, k = packed[:, :, :8], packed[:, :, 8:11]
    want_q, want_k = focus.rope(plan, q.contiguous(), k.contiguous(), offset=5)
    got_q, got_k = focus.rope(plan, q, k, offset=5)
    assert torch.equal(got_q, want_q) and torch.equal(got_k, want_k)
    assert torch.equal(focus.rope(plan, q, offset=5), want_q)
    # rows at odd element addresses, gaps between them
    wide = torch.zeros(2, 9, 8, 131, device="cuda", dtype=dtype)
    wide[..., 1:129] = q
    out = torch.full((2, 9, 8, 133), 7.0, device="cuda", dtype=dtype)
    focus.rope(plan, wide[..., 1:129], offset=5, out=out[..., 3:131])
    # the vector and the element path multiply and add alike
    assert torch.equal(out[..., 3:131], want_q)
    assert bool((out[..., :3] == 7).all()) and bool((out[..., 131:] == 7).all())
    # in place
    rest = packed[:, :, 11:].clone()
    focus.rope(plan, q, k, offset=5, out=q, out_k=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(packed[:, :, 11:], rest)


def test_rotation_backward_is_the_transposed_map():
    """<rope(x), g> = <x, rope_bwd(g)>, and differences of the forward in fp32."""
    plan = focus.Rope(dim=96, layout="half", scaling="by_parts", factor=4.0)
    x, g = randn(1, 40, 3, 128, seed=2, dtype=torch.float32).cuda(), randn(1, 40, 3, 128, seed=3, dtype=torch.float32).cuda()
    y, dx = focus.rope(plan, x, offset=100), focus.rope_bwd(plan, g, offset=100)
    a, b = (y.double() * g.double()).sum().item(), (x.double() * dx.double()).sum().item()
    assert abs(a - b) <= 2.0 ** -19 * (y.double().abs() * g.double().abs()).sum().item()
    # d <rope(x), g> / dx of a few elements: the map is linear, so a difference of any size does
    for at in [(0, 0, 0, 0), (0, 7, 1, 47), (0, 39, 2, 48), (0, 20, 0, 95), (0, 20, 0, 96), (0, 3, 2, 127)]:
        x2 = x.clone()
        x2[at] += 4.0
        dy = focus.rope(plan, x2, offset=100).double() - y.double()
        num = (dy * g.double()).sum().item() / (x2[at].item() - x[at].item())
        assert abs(num - dx[at].item()) <= 2.0 ** -16 * 8


def test_rotation_nan_and_infinity_stay_in_their_pair():
    plan = focus.Rope(dim=64)
    for dtype in (torch.bfloat16, torch.float32):
        x = randn(1, 3, 2, 128, seed=4, dtype=dtype)
        want = focus.rope(plan, x.cuda())
        x[0, 1, 0, 5], x[0, 1, 1, 100], x[0, 2, 0, 127] = math.nan, math.inf, math.nan
        got = focus.rope(plan, x.cuda())
        same = torch.ones(1, 3, 2, 128, dtype=torch.bool)
        for i in ((0, 1, 0, 5), (0, 1, 0, 37), (0, 1, 1, 100), (0, 2, 0, 127)):
            same[i] = False
        assert torch.equal(got.cpu()[same], want.cpu()[same])
        assert got[0, 1, 0, 5].isnan() and got[0, 1, 0, 37].isnan()
        assert got[0, 1, 1, 100] == math.inf and got[0, 2, 0, 127].isnan()


# ------------------------------------------------------------------------------ cache --
def cache_params(**kw):
    base = dict(B=2, cap=40, H=8, H_kv=2, d_head=128, R=1, K=4, top_k=2, w=8, format="bf16")
    base.update(kw)
    return focus.CacheParams(**base)


def filled_cache(p, seed):
    """A cache that holds tokens everywhere, on the GPU."""
    c = focus.KVCache.empty(p)
    x = randn(2, p.B, p.cap, p.H_kv, p.d_head, seed=seed, dtype=torch.float32)
    if p.format == "bf16":
        c.k.copy_(x[0].to(torch.bfloat16)), c.v.copy_(x[1].to(torch.bfloat16))
    else:
        unit = 140.0 if p.format == "e4m3" else 40.0
        for t, src in ((c.k, x[0]), (c.v, x[1])):
            codes = (src * unit).clamp(-127, 127).round() if p.format == "int8" else (src * unit).clamp(-448, 448)
            t.copy_(codes.to(t.dtype))
        g = torch.Generator().manual_seed(seed)
        for t in (c.k_scale, c.v_scale):
            t.copy_((torch.rand(t.shape, generator=g) + 0.5) / unit)
    c.mask.copy_(random_masks(seed, p.K, p.top_k, p.B, p.R, p.cap))
    return c


def raw(t):
    return t.view(torch.uint8).cpu() if t.dtype != torch.float32 else t.cpu()


def tensors(c):
    return [x for x in (c.k, c.v, c.k_scale, c.v_scale, c.mask) if x is not None]


WRITES = [
    dict(T=1, start=[0, 39]), dict(T=5, start=[35, 0]), dict(T=7, start=[3, 30], count=[0, 7]),
    dict(T=9, start=[10, 10], count=[9, 4], rope=dict(dim=128)), dict(T=3, start=[1, 2], rope=dict(dim=128, layout="interleaved")),
    dict(T=6, start=[20, 0], rope=dict(dim=64), positions=True, H_kv=5, H=5),
    dict(T=4, start=[4, 5], rope=dict(dim=38), H_kv=3, H=3, R=3),
    dict(T=4, start=[4, 5], rope=dict(dim=30, layout="interleaved"), d_head=64, H_kv=12, H=12),
    dict(T=11, start=[0, 29], rope=dict(dim=64, scaling="by_parts", factor=4.0), d_head=64, H_kv=1, H=4),
    dict(T=40, start=[0, 0], H_kv=8, R=8, rope=dict(dim=128), packed=True),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_cache_write_and_read(fmt, case):
    kw = dict(WRITES[case])
    T, start, count, rope = kw.pop("T"), kw.pop("start"), kw.pop("count", None), kw.pop("rope", None)
    given, packed = kw.pop("positions", False), kw.pop("packed", False)
    p = cache_params(format=fmt, **kw)
    c = filled_cache(p, case)
    old = [t.clone() for t in tensors(c)]
    if packed:
        both = randn(p.B, T, p.H + 2 * p.H_kv, p.d_head, seed=case).cuda()
        k, v = both[:, :, p.H:p.H + p.H_kv], both[:, :, p.H + p.H_kv:]
    else:
        k, v = randn(p.B, T, p.H_kv, p.d_head, seed=case).cuda(), randn(p.B, T, p.H_kv, p.d_head, seed=case + 9).cuda()
    mask = random_masks(case + 70, p.K, p.top_k, p.B, p.R, T).cuda()
    n = count or [T] * p.B
    pos = torch.tensor(start)[:, None] + torch.arange(T)
    if given:
        pos = torch.randint(0, 1 << 20, (p.B, T), generator=torch.Generator().manual_seed(case))
    plan = None if rope is None else focus.Rope(**rope)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    focus.cache_write(p, c, k, v, mask, torch.tensor(start, **i32), None if count is None else torch.tensor(n, **i32),
                      rope=plan, positions=pos.to(torch.int32).cuda() if given else None, status=status)
    assert focus.get_status(status) == 0
    # every other slot keeps its contents
    written = torch.zeros(p.B, p.cap, dtype=torch.bool)
    for b in range(p.B):
        written[b, start[b]:start[b] + n[b]] = True
    for new, was in zip(tensors(c), old):
        same = (raw(new) == raw(was))
        if new.dim() == 4:
            assert bool(same.view(p.B, p.cap, -1).all(-1)[~written].all())
        else:
            same = same.view(p.B, new.shape[1], p.cap, -1).all(-1)
            assert bool(same[(~written)[:, None].expand_as(same)].all())
    held = [ref.dequantise(c.k, c.k_scale), ref.dequantise(c.v, c.v_scale)]
    for b in range(p.B):
        at = slice(start[b], start[b] + n[b])
        assert torch.equal(c.mask[b, :, at].cpu(), mask[b, :, :n[b]].cpu())
        for i, (x, scale) in enumerate(((k, c.k_scale), (v, c.v_scale))):
            want, mag = x[b:b + 1, :n[b]].cpu().double(), torch.zeros(())
            if i == 0 and plan is not None:
                r = dict(rope)
                want, mag = ref.rotate(x[b:b + 1, :n[b]].cpu(), pos[b:b + 1, :n[b]], r.pop("dim"), r.pop("layout", "half"), **r)
            want, mag = want[0], 2.0 ** -20 * mag
            got = held[i][b, at]
            if fmt == "bf16":
                assert bool(((got - want).abs() <= u(torch.bfloat16) * want.abs() * (plan is not None and i == 0) + mag).all())
                continue
            unit = want.abs().amax(-1, keepdim=True) / ref.MAX_CODE[fmt]
            sc = scale[b, :, at].t().cpu().double()[..., None]
            assert bool(((sc - unit).abs() <= 2.0 ** -22 * unit + (mag.amax() if mag.dim() else 0) / ref.MAX_CODE[fmt]).all())
            step = 0.5 * sc if fmt == "int8" else torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * sc)
            assert bool(((got - want).abs() <= step * (1 + 2.0 ** -16) + 2 * mag + 2.0 ** -20 * want.abs()).all())
    # read back: codes times scales rounded once, zeros behind a sequence's end
    rk, rv = focus.cache_read(p, c, T, torch.tensor(start, **i32), None if count is None else torch.tensor(n, **i32),
                              status=status)
    assert focus.get_status(status) == 0
    for got, h in ((rk, held[0]), (rv, held[1])):
        for b in range(p.B):
            want = h[b, start[b]:start[b] + n[b]]
            err = (got[b, :n[b]].cpu().double() - want).abs()
            assert bool((err <= (u(torch.bfloat16) + 2.0 ** -23) * want.abs()).all())
            assert bool((got[b, n[b]:] == 0).all())


def test_cache_rows_of_zeros_tiny_and_not_finite_values():
    p0 = cache_params(B=1, cap=8, H_kv=2, H=2)
    x = randn(1, 6, 2, 128, seed=5).float()
    x[0, 0] = 0.0
    x[0, 1] = 2.0 ** -110
    x[0, 2, 0, 17] = math.nan
    x[0, 3, 1, 99] = -math.inf
    x[0, 4] *= 1e37 / 4
    x[0, 5] *= 2.0 ** -90
    x = x.to(torch.bfloat16).cuda()
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    for fmt in ("e4m3", "int8"):
        p = dataclasses.replace(p0, format=fmt)
        c = focus.KVCache.empty(p)
        focus.cache_write(p, c, x, x, None, start)
        k, v = focus.cache_read(p, c, 6)
        assert bool((k[0, 0] == 0).all()) and bool((k[0, 1] == 0).all()) and bool((c.k_scale[0, :, :2] == 0).all())
        assert bool(k[0, 2, 0].isnan().all()) and bool(v[0, 3, 1].isnan().all())
        assert bool(k[0, 2, 1].isfinite().all()) and bool(v[0, 3, 0].isfinite().all())
        assert bool((c.k.view(torch.uint8)[0, 2, 0] == 0).all())
        err = (k[0, 4:].double() - x[0, 4:].double()).abs().amax(-1) / x[0, 4:].double().abs().amax(-1)
        assert err.max().item() <= (2.0 ** -4 if fmt == "e4m3" else 0.5 / 127) + 2.0 ** -8


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("H_kv,d", [(1, 64), (1, 128), (2, 64), (3, 64), (2, 128), (7, 64)])
def test_cache_of_few_heads_and_many_tokens(fmt, H_kv, d):
    """The same bits as head by head in a cache of many heads, where a warp takes one token."""
    B, T, wide = 3, 1201, 16
    p = cache_params(B=B, cap=T + 30, H=H_kv, H_kv=H_kv, d_head=d, K=8, R=H_kv, format=fmt)
    pw = dataclasses.replace(p, H=wide, H_kv=wide, R=1)
    k, v = randn(B, T, H_kv, d, seed=1).cuda(), randn(B, T, H_kv, d, seed=2).cuda()
    mask = random_masks(3, 8, 2, B, H_kv, T).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    start, count = torch.tensor([0, 29, 7], **i32), torch.tensor([T, T, 600], **i32)
    c, cw = focus.KVCache.empty(p), focus.KVCache.empty(pw)
    plan = focus.Rope(dim=d)
    rep = lambda x: torch.nn.functional.pad(x, (0, 0, 0, wide - H_kv))
    focus.cache_write(p, c, k, v, mask, start, count, rope=plan)
    focus.cache_write(pw, cw, rep(k), rep(v), None, start, count, rope=plan)
    assert torch.equal(raw(c.k), raw(cw.k)[:, :, :H_kv]) and torch.equal(raw(c.v), raw(cw.v)[:, :, :H_kv])
    if fmt != "bf16":
        assert torch.equal(c.k_scale, cw.k_scale[:, :H_kv]) and torch.equal(c.v_scale, cw.v_scale[:, :H_kv])
    for b, (s, n) in enumerate(((0, T), (29, T), (7, 600))):
        assert torch.equal(c.mask[b, :, s:s + n], mask[b, :, :n])
        assert not bool(c.mask[b, :, :s].any()) and not bool(c.mask[b, :, s + n:].any())
    for x, y in zip(focus.cache_read(p, c, T, start, count), focus.cache_read(pw, cw, T, start, count)):
        assert torch.equal(x, y[:, :, :H_kv])
        assert bool((x[2, 600:] == 0).all())


def test_cache_slots_outside_are_reported_and_not_touched():
    """Device-side refusals: tokens without a slot and counts outside [0, T] set the status
    word; nothing outside [start, start + count) changes, reads give zeros."""
    for fmt in ("bf16", "int8"):
        p = cache_params(B=3, cap=10, format=fmt)
        x = randn(3, 4, 2, 128, seed=8).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        for start, count, rows in (([8, -2, 0], None, [(8, 10), (0, 2), (0, 4)]),
                                   ([10, 2147483647, -2147483648], None, [(0, 0)] * 3),
                                   ([0, 0, 0], [5, -1, 2], [(0, 4), (0, 0), (0, 2)])):
            c = filled_cache(p, 3)
            old = [raw(t).clone() for t in tensors(c)]
            status = torch.zeros(1, **i32)
            cnt = None if count is None else torch.tensor(count, **i32)
            focus.cache_write(p, c, x, x, None, torch.tensor(start, **i32), cnt, status=status)
            assert focus.get_status(status) == -6
            keep = torch.ones(3, 10, dtype=torch.bool)
            for b, (lo, hi) in enumerate(rows):
                keep[b, lo:hi] = False
            for new, was in zip((c.k, c.v), old):
                same = (raw(new) == was).view(3, 10, -1).all(-1)
                assert bool(same[keep].all()) and not bool(same[~keep].any())
            status.zero_()
            k, _ = focus.cache_read(p, c, 4, torch.tensor(start, **i32), cnt, status=status)
            assert focus.get_status(status) == -6
            for b in range(3):
                for t in range(4):
                    inside = 0 <= start[b] + t < 10 and t < (4 if count is None else count[b])
                    assert bool((k[b, t] != 0).any()) == inside


# --------------------------------------------------------------------------- decoding --
TREES = {
    "one_token": dict(T=1, lens=[37, 12]),
    "one_token_empty_cache": dict(T=1, lens=[0, 1], w=1),
    "mha64": dict(T=1, lens=[39, 7, 0], B=3, H=12, H_kv=12, d_head=64, K=4, top_k=2, w=5),
    "mqa16": dict(T=3, lens=[300, 256], cap=400, H=16, H_kv=1, w=33, R=1, K=8, top_k=2),
    "chain5": dict(T=5, lens=[100, 130], cap=140, R=2, w=10),
    "tree7_w1": dict(T=7, lens=[64, 33], cap=80, tree=True, w=1, K=8, top_k=1),
    "tree16": dict(T=16, lens=[500, 31], cap=520, tree=True, K=8, top_k=2, w=40, R=2),
    "tree64": dict(T=64, lens=[200, 1], cap=264, tree=True, K=4, top_k=1, w=20),
    "tree33_gqa3": dict(T=33, lens=[90], B=1, cap=130, tree=True, H=6, H_kv=2, d_head=64, w=7, R=2),
    "tree9_window_covers_all": dict(T=9, lens=[50, 60], cap=70, tree=True, w=1 << 30),
    "tree12_dead_rows": dict(T=12, lens=[70, 0], cap=90, tree=True, dead=True, w=3, K=8, top_k=1),
    "one_group": dict(T=6, lens=[300], B=1, cap=310, tree=True, K=1, top_k=1, w=2),
    "K32": dict(T=10, lens=[400], B=1, cap=410, tree=True, K=32, top_k=4, w=16),
    "no_masks": dict(T=10, lens=[400], B=1, cap=410, tree=True, zero_masks=True, w=16),
    "ragged_40": dict(T=2, B=40, lens=[(b * 53) % 200 for b in range(40)], cap=202, w=9, H=2, H_kv=1, d_head=64),
    "long_one": dict(T=4, B=3, lens=[3000, 3, 0], cap=3100, w=100, tree=True, H=4, H_kv=2, d_head=64),
    "long_tree": dict(T=24, B=3, lens=[3000, 700, 0], cap=3100, w=100, tree=True, H=8, H_kv=2, K=8, top_k=1),
    "ragged_tree": dict(T=9, B=20, lens=[(b * 37) % 150 for b in range(20)], cap=160, w=9, tree=True, H=4, H_kv=1, d_head=64),
    "sparse_tree": dict(T=17, lens=[2500], B=1, cap=2600, w=1, tree=True, H=2, H_kv=1, K=32, top_k=1),
    "wide_tree": dict(T=64, lens=[1500], B=1, cap=1600, w=30, tree=True, H=4, H_kv=1, K=4, top_k=1),
    "wide_tree64": dict(T=40, lens=[1201, 700], cap=1300, w=30, tree=True, H=6, H_kv=1, d_head=64, K=4, top_k=2),
    "sparse_wide": dict(T=17, lens=[1300], B=1, cap=1400, w=5, tree=True, H=8, H_kv=1, K=32, top_k=1),
    "rows_300": dict(T=50, lens=[90, 600], cap=700, w=64, tree=True, H=6, H_kv=1, K=8, top_k=2),
    "scale": dict(T=4, lens=[100, 20], cap=120, softmax_scale=0.5, tree=True),
}


def tree_case(name, fmt, seed=0, big=False):
    """big: in a cache of so many slots that more than 16 rows go to the tensor-core kernel."""
    kw = dict(TREES[name])
    T, lens, is_tree = kw.pop("T"), kw.pop("lens"), kw.pop("tree", False)
    dead, zero = kw.pop("dead", False), kw.pop("zero_masks", False)
    kw.setdefault("B", len(lens))
    p = cache_params(format=fmt, **kw)
    if big:
        p = dataclasses.replace(p, cap=max(p.cap, 32 * 6500 // (p.B * p.H_kv) + 7))
    c = filled_cache(p, seed + 11)
    if zero:
        c.mask.zero_()
    q = randn(p.B, T, p.H, p.d_head, seed=seed + 1)
    rng = random.Random(seed)
    words = [ref.random_tree(rng, T) if is_tree else [(2 << t) - 1 for t in range(T)] for _ in lens]
    if dead:
        words = [[0 if t in (0, 5, T - 1) else x for t, x in enumerate(row)] for row in words]
    return p, c, q, T, lens, words, is_tree


def check_tree(p, c, q, lens, words, o, lse, fmt):
    n = max(lens) + q.shape[1]
    kv = [ref.dequantise(x[:, :n], None if y is None else y[:, :, :n]) for x, y in ((c.k, c.k_scale), (c.v, c.v_scale))]
    want, want_lse, m, s, z = ref.decode_tree(q, *kv, c.mask[:, :, :n], lens, words, w=p.w, R=p.R, scale=p.scale,
                                           vs=None if c.v_scale is None else c.v_scale[:, :, :n].cpu())
    ds = p.d_head * 2.0 ** -22 * s
    up = u(torch.bfloat16 if fmt == "bf16" else torch.float16)
    bound = (up + 4 * ds.transpose(1, 2)[..., None] + 2.0 ** -18) * m + u(torch.bfloat16) * want.abs() + 2.0 ** -28 * z
    err = (o.cpu().double() - want).abs()
    empty = want_lse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty)
    assert bool((o.cpu()[empty.transpose(1, 2)] == 0).all())
    lerr = (lse.cpu().double() - want_lse).abs()[~empty]
    lbound = (2 * ds + 2.0 ** -18 * want_lse.abs().clamp(min=1))[~empty]
    ratio = float((err / bound.clamp(min=1e-30)).max()), float((lerr / lbound).max()) if len(lerr) else 0.0
    print("max err / bound: o %.2f lse %.2f" % ratio)
    assert ratio[0] <= 1.0, (ratio, [(i.tolist(), err[tuple(i)].item(), want[tuple(i)].item(), m[tuple(i)].item(), z[tuple(i)].item())
                                     for i in (err > bound).nonzero()[:8]])
    assert bool((lerr <= lbound).all()), ratio


ROWS = {n: kw["T"] * kw.get("H", 8) // kw.get("H_kv", 2) for n, kw in TREES.items()}
SIZES = [(n, False) for n in TREES] + [(n, True) for n in TREES if ROWS[n] > 16]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("name,big", SIZES)
def test_decode_tree_matches_the_definition(name, big, fmt):
    p, c, q, T, lens, words, is_tree = tree_case(name, fmt, big=big)
    ws = torch.empty(focus.decode_tree_workspace_size(p, T), dtype=torch.uint8, device="cuda")
    tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda") if is_tree else None
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = focus.decode_tree(p, q.cuda(), c, n, tree, ws=ws)
    assert focus.get_status(ws) == 0
    check_tree(p, c, q, lens, words, o, lse, fmt)
    # the same call twice gives the same bits; a NULL tree is the chain
    o2, lse2 = focus.decode_tree(p, q.cuda(), c, n, tree)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if not is_tree:
        chain = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda")
        o3, lse3 = focus.decode_tree(p, q.cuda(), c, n, chain)
        assert torch.equal(o, o3) and torch.equal(lse, lse3)
    assert focus.decode_tree(p, q.cuda(), c, n, tree, want_lse=False)[1] is None


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_decode_tree_ignores_what_it_must_not_see(fmt, big):
    """NaN and infinities in slots behind the drafted tokens, in keys whose masks do not
    meet a row's and in other branches of the tree reach no row that does not see them."""
    p, c, q, T, lens, words, _ = tree_case("tree16", fmt, big=big)
    lens, words = [500, 31], [[1 << t | 1 for t in range(T)] for _ in lens]   # leaves of one root
    tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean, clean_lse = focus.decode_tree(p, q.cuda(), c, n, tree)

    def spoil(b, j, value):
        if fmt == "bf16":
            c.k[b, j] = value
            c.v[b, j] = value
        else:
            c.k_scale[b, :, j] = value
            c.v_scale[b, :, j] = value

    spoil(0, slice(lens[0] + T, p.cap), math.nan)
    spoil(1, slice(lens[1] + T, p.cap), math.inf)
    o, lse = focus.decode_tree(p, q.cuda(), c, n, tree)
    assert torch.equal(o, clean) and torch.equal(lse, clean_lse)
    # a leaf's own key: only that leaf's rows change
    spoil(0, lens[0] + 3, math.nan)
    # a far key with one group: rows that do not have it keep their values
    c.mask[0, :, 100] = 4
    c.mask[0, :, lens[0]:lens[0] + T] = 3
    c.mask[0, 1, lens[0] + 7] = 6
    ref_o, ref_lse = focus.decode_tree(p, q.cuda(), c, n, tree)
    spoil(0, 100, math.inf if fmt == "bf16" else math.nan)
    o, lse = focus.decode_tree(p, q.cuda(), c, n, tree)
    per = p.H // p.R
    for b in range(2):
        for t in range(T):
            for r in range(p.R):
                got = o[b, t, r * per:(r + 1) * per]
                if b == 0 and (t == 3 or (t == 7 and r == 1)):
                    assert bool((~got.isfinite()).all())
                else:
                    want = ref_o[b, t, r * per:(r + 1) * per]
                    assert bool(got.isfinite().all())
                    # such a row is computed again key by key: fp32 throughout
                    assert bool(((got.float() - want.float()).abs() <= 2.0 ** -6).all())
                    got_l, want_l = (x[b, r * per:(r + 1) * per, t].double() for x in (lse, ref_lse))
                    # A scale that is no number has its tile's reference m taken key by key, not by
                    # one power of two: the terms 2^(s - m) are rounded anew on both sides.  Terms
                    # that count have |s - m| < 32, rounded by 2^-20, times ln 2; the exponential
                    # adds 2^-22, a sum through at most 32 additions 2^-19, m + log2(l) below 64
                    # 2^-19: twice their sum is below 2^-16.  bf16 caches have no scales.
                    assert bool(((got_l - want_l).abs() <= (0.0 if fmt == "bf16" else 2.0 ** -16)).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name,big", [("chain5", False), ("chain5", True), ("tree16", False), ("tree16", True),
                                      ("mha64", False), ("rows_300", True)])
def test_decode_tree_scales_far_apart(name, big, fmt):
    """V scales of very different sizes, zeros among them, in keys that rows see and in keys
    that they do not: no row loses its own keys' digits to another key's scale."""
    p, c, q, T, lens, words, is_tree = tree_case(name, fmt, seed=5, big=big)
    g = torch.Generator().manual_seed(1)
    size = torch.randint(-24, 24, c.v_scale.shape, generator=g).double()
    size[:, :, ::3] = 0
    c.v_scale.copy_(c.v_scale.cpu() * torch.exp2(size).float())
    c.v_scale[:, :, 5::11] = 0.0
    c.k_scale[:, :, 7::13] = 0.0
    # a key of a group of its own, far larger than all others: nobody sees it
    c.mask[:, :, 2] = 1 << 20
    c.v_scale[:, :, 2] = 1e20
    tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda") if is_tree else None
    o, lse = focus.decode_tree(p, q.cuda(), c, torch.tensor(lens, dtype=torch.int32, device="cuda"), tree)
    check_tree(p, c, q, lens, words, o, lse, fmt)


def test_decode_tree_logits_that_grow_and_fall():
    """Logits that rise by hundreds along the sequence, and fall again: the reference of the
    exponentials moves many times."""
    for name, big in (("tree16", False), ("tree16", True), ("chain5", False), ("one_token", False), ("rows_300", True)):
        for fmt in ("bf16", "int8"):
            p, c, q, T, lens, words, is_tree = tree_case(name, fmt, seed=6, big=big)
            up = torch.linspace(0, 30, max(lens) + T)
            up = torch.nn.functional.pad(torch.minimum(up, 40 - up), (0, p.cap - max(lens) - T))
            if fmt == "bf16":
                c.k.copy_((q.mean((0, 1, 2)) * up[:, None]).to(torch.bfloat16)[None, :, None].expand(c.k.shape))
            else:
                c.k_scale.copy_(c.k_scale.cpu() * up)
            tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda") if is_tree else None
            o, lse = focus.decode_tree(p, q.cuda(), c, torch.tensor(lens, dtype=torch.int32, device="cuda"), tree)
            check_tree(p, c, q, lens, words, o, lse, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name,big", [("one_token", False), ("chain5", False), ("tree16", True)])
def test_decode_tree_queries_at_the_ends_of_the_range(name, big, fmt):
    """Queries near the largest and below the smallest normal bf16 number, against key scales
    that bring the logits back: rows are scaled by powers of two, exactly."""
    for e in (126, -127):
        p, c, q, T, lens, words, is_tree = tree_case(name, fmt, seed=8, big=big)
        q = (q.double().clamp(-3.9, 3.9) * 2.0 ** e).to(torch.bfloat16)
        half = 2.0 ** (-60 if e > 0 else 60)
        c.k_scale.mul_(half)
        p = dataclasses.replace(p, softmax_scale=2.0 ** -e / half / math.sqrt(p.d_head))
        tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda") if is_tree else None
        o, lse = focus.decode_tree(p, q.cuda(), c, torch.tensor(lens, dtype=torch.int32, device="cuda"), tree)
        check_tree(p, c, q, lens, words, o, lse, fmt)


def test_decode_tree_of_queries_that_are_not_finite():
    """A NaN or an infinity in a query shows in its own row only."""
    for name, big in (("one_token", False), ("chain5", False), ("tree16", True), ("rows_300", True)):
        for fmt in ("bf16", "int8"):
            p, c, q, T, lens, words, is_tree = tree_case(name, fmt, seed=9, big=big)
            tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda") if is_tree else None
            n = torch.tensor(lens, dtype=torch.int32, device="cuda")
            want, want_lse = focus.decode_tree(p, q.cuda(), c, n, tree)
            hit = torch.zeros(q.shape[:3], dtype=torch.bool)
            for i, value in enumerate((math.nan, math.inf, -math.inf)):
                q[0, (3 * i) % T, i % p.H, 7] = value
                hit[0, (3 * i) % T, i % p.H] = True
            got, lse = focus.decode_tree(p, q.cuda(), c, n, tree)
            assert torch.equal(got.cpu()[~hit], want.cpu()[~hit])
            assert torch.equal(lse.transpose(1, 2).cpu()[~hit], want_lse.transpose(1, 2).cpu()[~hit])
            assert bool(got.cpu()[hit].isnan().all(-1).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("H,H_kv,d", [(1, 0, 64), (1, 1, 64), (2, 1, 64), (1, 0, 128), (1, 1, 128), (3, 2, 64)])
def test_rotation_of_few_heads_and_many_tokens(H, H_kv, d, layout, dtype):
    """The same bits as in a call of many heads, where a warp takes one token."""
    B, N = 3, 1701
    plan = focus.Rope(dim=d if H > 1 else d // 2, layout=layout, scaling="by_parts", factor=4.0)
    q = randn(B, N, H, d, seed=1, dtype=dtype).cuda()
    k = randn(B, N, H_kv, d, seed=2, dtype=dtype).cuda() if H_kv else None
    pos = torch.randint(-5, 1 << 20, (B, N), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    for call, kw in ((focus.rope, dict(offset=77)), (focus.rope_bwd, dict(positions=pos))):
        wide = call(plan, torch.cat([q] * 16, 2), **kw)
        got = call(plan, q, k, **kw)
        assert torch.equal(got[0] if H_kv else got, wide[:, :, :H])
        if H_kv:
            assert torch.equal(got[1], call(plan, torch.cat([k] * 16, 2), **kw)[:, :, :H_kv])


def test_rotation_of_broadcast_views():
    """One key head shown to all, as an expanded view: like its copies.  Outputs that share
    elements are refused."""
    plan = focus.Rope(dim=64)
    q, one = randn(2, 5, 4, 128, seed=1).cuda(), randn(2, 5, 1, 128, seed=2).cuda()
    k = one.expand(2, 5, 4, 128)
    want, got = focus.rope(plan, q, k.contiguous()), focus.rope(plan, q, k)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(focus.FocusError):
        focus.rope(plan, q, k, out_k=k)
    with pytest.raises(focus.FocusError):
        focus.rope(plan, q, out=one.expand(2, 5, 4, 128))


def test_calls_whose_tensors_overlap_are_refused():
    p = cache_params(B=1, cap=40)
    c = focus.KVCache.empty(p)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(focus.FocusError):
        focus.cache_write(p, c, c.k[:, 3:6], c.v[:, 3:6], None, n)
    with pytest.raises(focus.FocusError):
        focus.cache_read(p, c, 3, out=(c.k[:, :3], c.v[:, :3]))
    q = randn(1, 2, p.H, p.d_head).cuda()
    with pytest.raises(focus.FocusError):
        focus.decode_tree(p, q, c, n, out=q)


def test_decode_tree_refuses_lengths_outside_the_cache():
    p, c, q, T, lens, words, _ = tree_case("ragged_40", "int8")
    n = torch.tensor(lens, dtype=torch.int32)
    want, want_lse = focus.decode_tree(p, q.cuda(), c, n.cuda())
    bad = n.clone()
    bad[3], bad[17], bad[39] = -1, p.cap - T + 1, 2147483647
    ws = torch.empty(focus.decode_tree_workspace_size(p, T), dtype=torch.uint8, device="cuda")
    o, lse = focus.decode_tree(p, q.cuda(), c, bad.cuda(), ws=ws)
    assert focus.get_status(ws) == -6
    hit = torch.zeros(p.B, dtype=torch.bool)
    hit[[3, 17, 39]] = True
    assert bool((o.cpu()[hit] == 0).all()) and bool((lse.cpu()[hit] == -math.inf).all())
    err = (o.cpu()[~hit].float() - want.cpu()[~hit].float()).abs().max()
    assert err.item() <= 2.0 ** -5 and bool(torch.isfinite(lse.cpu()[~hit]).all())
    focus.decode_tree(p, q.cuda(), c, n.cuda(), ws=ws)
    assert focus.get_status(ws) == 0


def test_decode_tree_of_one_token_agrees_with_decode():
    """The step of one token over a bf16 cache is focus_decode on the same tokens."""
    import synth
    wl = synth.WORKLOADS["tiny"].replace(B=1, N=2000, H=8, H_kv=2, d_head=128, K=8, top_k=2, w=100)
    x = synth.make_inputs(wl, seed=21, device="cuda")
    p = focus.Params.from_workload(wl)
    mask, _ = focus.route(p, x["r"], x["C"])
    o, lse = focus.decode(p, x["q"][:, -1].contiguous(), x["k"], x["v"], mask)
    pc = cache_params(B=1, cap=2000, H=8, H_kv=2, K=8, top_k=2, w=100)
    c = focus.KVCache(x["k"], x["v"], None, None, mask)
    o2, lse2 = focus.decode_tree(pc, x["q"][:, -1:].contiguous(), c, torch.tensor([1999], dtype=torch.int32, device="cuda"))
    assert (o.float() - o2[:, 0].float()).abs().max().item() <= 2.0 ** -7
    assert (lse - lse2[:, :, 0]).abs().max().item() <= 1e-5


# --------------------------------------------------- the operators together, as in use --
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_prompt_draft_commit_and_next_step(fmt):
    """A prompt enters the cache (rotated, routed), a tree is drafted and decoded, the
    accepted path is committed by writing it again, and the next draft decodes: each step
    against the definition on what the cache holds; the committed rows equal those of a
    cache that was fed the path directly."""
    B, H, H_kv, d, K, top_k, w = 2, 8, 2, 128, 4, 2, 16
    p = cache_params(B=B, cap=160, H=H, H_kv=H_kv, K=K, top_k=top_k, w=w, format=fmt)
    plan = focus.Rope(dim=d)
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)
    C = torch.randn(K, 16, generator=g).cuda()

    def tokens(T, seed):
        x = [randn(B, T, h, d, seed=seed + i).cuda() for i, h in enumerate((H, H_kv, H_kv))]
        r = torch.randn(B, T, 1, 16, generator=torch.Generator().manual_seed(seed)).cuda()
        pr = focus.Params(B=B, N=T, H=H, H_kv=H_kv, d_head=d, R=1, K=K, top_k=top_k, w=w)
        return (*x, focus.route(pr, r, C)[0])

    lens = [100, 61]
    q, k, v, mask = tokens(100, 40)
    c = focus.KVCache.empty(p)
    focus.cache_write(p, c, k, v, mask, torch.zeros(B, **i32), torch.tensor(lens, **i32), rope=plan)
    rng = random.Random(9)
    T = 12
    words = [ref.random_tree(rng, T, 4) for _ in range(B)]
    q, k, v, mask = tokens(T, 50)
    depth = torch.tensor([[bin(x).count("1") - 1 for x in row] for row in words])
    n = torch.tensor(lens, **i32)
    pos = (torch.tensor(lens)[:, None] + depth).to(torch.int32).cuda()
    focus.cache_write(p, c, k, v, mask, n, rope=plan, positions=pos)
    qr = focus.rope(plan, q, positions=pos)
    tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda")
    o, lse = focus.decode_tree(p, qr, c, n, tree)
    check_tree(p, c, qr.cpu(), lens, words, o, lse, fmt)
    # accept the path to the last token: its tokens again, in order, at consecutive slots
    path = [[u for u in range(T) if words[b][T - 1] >> u & 1] for b in range(B)]
    took = [len(x) for x in path]
    rows = torch.zeros(B, max(took), dtype=torch.long)
    for b in range(B):
        rows[b, :took[b]] = torch.tensor(path[b])
    pick = torch.arange(B)[:, None], rows
    accepted = [k.cpu()[pick].cuda(), v.cpu()[pick].cuda(), mask.cpu().transpose(1, 2)[pick].transpose(1, 2).contiguous().cuda()]
    focus.cache_write(p, c, *accepted, n, torch.tensor(took, **i32), rope=plan)
    fresh = focus.KVCache.empty(p)
    _, k0, v0, mask0 = tokens(100, 40)
    focus.cache_write(p, fresh, k0, v0, mask0, torch.zeros(B, **i32), torch.tensor(lens, **i32), rope=plan)
    focus.cache_write(p, fresh, *accepted, n, torch.tensor(took, **i32), rope=plan)
    for b in range(B):
        end = lens[b] + took[b]
        assert torch.equal(raw(c.k)[b, :end], raw(fresh.k)[b, :end]) and torch.equal(c.mask[b, :, :end], fresh.mask[b, :, :end])
    lens = [lens[b] + took[b] for b in range(B)]
    n = torch.tensor(lens, **i32)
    q, k, v, mask = tokens(1, 60)
    focus.cache_write(p, c, k, v, mask, n, rope=plan)
    qr = focus.rope(plan, q, positions=n[:, None].contiguous())
    o, lse = focus.decode_tree(p, qr, c, n)
    check_tree(p, c, qr.cpu(), lens, [[1]] * B, o, lse, fmt)
    # the prefix read back feeds the forward pass: the last row of it is the step's
    if fmt == "bf16":
        N = lens[0] + 1
        kk, vv = focus.cache_read(p, c, N)
        qq = randn(1, N, H, d, seed=77).cuda()
        qq[:, -1] = qr[:1, 0]
        pf = focus.Params(B=1, N=N, H=H, H_kv=H_kv, d_head=d, R=1, K=K, top_k=top_k, w=w)
        of, _ = focus.attn_fwd(pf, qq, kk[:1].contiguous(), vv[:1].contiguous(), mask=c.mask[:1, :, :N].contiguous())
        assert (of[0, -1].float() - o[0, 0].float()).abs().max().item() <= 2.0 ** -6


def test_step_in_a_graph_on_side_streams_and_two_graphs():
    """A serving step (write, rotate, decode) captured twice with workspaces of its own,
    replayed in turn on other inputs and lengths: equal to eager calls bit for bit."""
    p = cache_params(B=4, cap=700, H=8, H_kv=2, K=8, top_k=2, w=50, format="e4m3")
    plan = focus.Rope(dim=128)
    T = 3
    cache = filled_cache(p, 4)

    def step(x, stream=None):
        focus.cache_write(p, cache, x["k"], x["v"], x["mask"], x["n"], rope=plan, stream=stream)
        q = focus.rope(plan, x["q"], positions=x["pos"], stream=stream)
        return focus.decode_tree(p, q, cache, x["n"], stream=stream)

    def inputs(seed):
        n = torch.randint(0, 690, (4,), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        return {"q": randn(4, T, 8, 128, seed=seed).cuda(), "k": randn(4, T, 2, 128, seed=seed + 1).cuda(),
                "v": randn(4, T, 2, 128, seed=seed + 2).cuda(), "mask": random_masks(seed, 8, 2, 4, 1, T).cuda(),
                "n": n.cuda(), "pos": (n[:, None] + torch.arange(T, dtype=torch.int32)).cuda()}

    x = inputs(100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = step(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(x)
        graphs.append((graph, out))
    again = step(x)
    assert torch.equal(on_side[0], again[0]) and torch.equal(on_side[1], again[1])
    for seed in (200, 300, 400):
        y = inputs(seed)
        for name in x:
            x[name].copy_(y[name])
        graph, out = graphs[seed // 100 % 2]
        graph.replay()
        got = [t.clone() for t in out]
        want = step(x)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_slots_behind_four_gigabytes(fmt):
    """Element offsets past 2^32 in the cache: the last sequence of a large one."""
    p = cache_params(B=3, cap=1 << 20, H=16, H_kv=16, d_head=128, K=1, top_k=1, w=4, format=fmt)
    c = focus.KVCache.empty(p)
    c.mask.zero_()
    T, at = 2, (1 << 20) - 12
    k, v = randn(3, 10, 16, 128, seed=1).cuda(), randn(3, 10, 16, 128, seed=2).cuda()
    n = torch.full((3,), at, dtype=torch.int32, device="cuda")
    focus.cache_write(p, c, k, v, None, n)
    rk, rv = focus.cache_read(p, c, 10, n)
    tol = 0.0 if fmt == "bf16" else 0.5 / 127 * 6 + 2.0 ** -6
    assert (rk.float() - k.float()).abs().max().item() <= tol and (rv.float() - v.float()).abs().max().item() <= tol
    q = randn(3, T, 16, 128, seed=3)
    o, lse = focus.decode_tree(p, q.cuda(), c, n + 8)
    # the window is all that is seen: the same tokens in a small cache
    ps = cache_params(B=3, cap=10, H=16, H_kv=16, d_head=128, K=1, top_k=1, w=4, format=fmt)
    cs = focus.KVCache(*[None if x is None else x for x in (
        c.k[:, at:at + 10].contiguous(), c.v[:, at:at + 10].contiguous(),
        None if c.k_scale is None else c.k_scale[:, :, at:at + 10].contiguous(),
        None if c.v_scale is None else c.v_scale[:, :, at:at + 10].contiguous(), c.mask[:, :, at:at + 10].contiguous())])
    check_tree(ps, cs, q, [8] * 3, [[1, 3]] * 3, o, lse, fmt)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one GPU")
def test_tensors_of_another_device():
    plan = focus.Rope(dim=128)
    x = randn(1, 4, 2, 128).to("cuda:1")
    assert torch.equal(focus.rope(plan, x).cpu(), focus.rope(plan, x.to("cuda:0")).cpu())
