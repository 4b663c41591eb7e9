"""Host-side checks of the rotary, cache and tree-decode entry points (no GPU needed):
the rotary plan against its definition, and refusals before anything is launched."""
import ctypes
import math

import pytest
import torch

import learned_centroid_gated_gb300 as focus
import serving_ref as ref

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="passes made-up device addresses; host-only check")
E = {v: k for k, v in focus.ERRORS.items()}
P = ctypes.c_void_p
OK = P(1 << 12)


@pytest.mark.parametrize("kw", [dict(dim=128), dict(dim=2), dict(dim=64, layout="interleaved", base=5e5),
                                dict(dim=100, scaling="linear", factor=3.0), dict(dim=128, scaling="ntk", factor=8.0),
                                dict(dim=2, scaling="ntk", factor=8.0),
                                dict(dim=128, scaling="by_parts", factor=32.0, orig_len=8192),
                                dict(dim=64, scaling="by_parts", factor=2.0, attn_factor=1.5, beta_slow=0.0)])
def test_rope_plan_is_the_definition(kw):
    plan = focus.Rope(**kw)._plan
    arg = {k: v for k, v in kw.items() if k != "layout"}
    f, g = ref.frequencies(**arg)
    for i in range(64):
        want = float(f[i]) / (2 * math.pi) * 2.0 ** 64 if i < kw["dim"] // 2 else 0.0
        assert abs(plan.turn[i] - want) <= 2.0 ** -50 * want + 1
    assert abs(plan.attn_factor - g) <= 2.0 ** -24 * g


def test_rope_positions_wrap_exactly():
    """pos * turn modulo 2^64 is the phase to 2^-30 of a turn for any 32-bit position."""
    plan = focus.Rope(dim=128)._plan
    f, _ = ref.frequencies(128)
    from fractions import Fraction
    for pos in (1, 12345, (1 << 20) + 1, (1 << 31) - 1, -(1 << 31), -7):
        for i in (0, 1, 17, 63):
            phase = (pos * plan.turn[i]) % (1 << 64) / 2.0 ** 64
            true = Fraction(float(f[i])) * pos / Fraction(2 * math.pi)
            true = float(true - math.floor(true))
            d = abs(phase - true)
            assert min(d, 1 - d) <= 2.0 ** -19 * 2.0 ** -32 * abs(pos) + 2.0 ** -21


@pytest.mark.parametrize("kw", [dict(dim=0), dict(dim=3), dict(dim=130), dict(dim=64, base=0.5), dict(dim=64, base=math.inf),
                                dict(dim=64, scaling="linear", factor=0.5), dict(dim=64, scaling="ntk", factor=math.nan),
                                dict(dim=64, scaling="by_parts", factor=2.0, orig_len=0), dict(dim=64, layout="other"),
                                dict(dim=64, scaling="by_parts", factor=2.0, beta_slow=40.0), dict(dim=64, scaling="x")])
def test_rope_plan_refusals(kw):
    with pytest.raises(focus.FocusError):
        focus.Rope(**kw)


def _rope(plan=None, dtype=0, B=1, N=4, H=2, H_kv=1, d=128, q=OK, k=OK, pos=None, qo=OK, ko=OK):
    plan = plan or focus.Rope(dim=64)._plan
    return focus._lib.focus_rope_apply(ctypes.addressof(plan), dtype, B, N, H, H_kv, d, q, None, k, None, pos, 0, 0, qo,
                                       None, ko, None, None)


@host_only
def test_rope_argument_errors():
    assert _rope(q=None) == _rope(qo=None) == _rope(ko=None) == E["FOCUS_ERR_INVALID_ARG"]
    assert _rope(B=0) == _rope(N=0) == _rope(H=0) == _rope(H_kv=0) == _rope(dtype=3) == E["FOCUS_ERR_INVALID_ARG"]
    assert _rope(d=96) == E["FOCUS_ERR_UNSUPPORTED"]
    assert _rope(plan=focus.Rope(dim=128)._plan, d=64) == E["FOCUS_ERR_INVALID_ARG"]
    assert _rope(B=1 << 20, N=1 << 20) == E["FOCUS_ERR_UNSUPPORTED"]
    assert _rope(q=P(4097)) == _rope(pos=P(4098)) == _rope(dtype=2, ko=P(4098)) == E["FOCUS_ERR_ALIGNMENT"]


def _cp(**kw):
    base = dict(B=2, cap=64, T=3, H=8, H_kv=2, d_head=128, R=1, K=4, top_k=2, w=16, format=0, softmax_scale=0.0)
    base.update(kw)
    return focus._CacheParams(*base.values())


def _write(p, k=OK, v=OK, mask=OK, start=OK, count=None, kc=OK, vc=OK, ks=None, vs=None, mc=OK, status=None, st=None,
           rope=None):
    return focus._lib.focus_cache_write(ctypes.byref(p), k, st, v, None, mask, start, count, rope, None, kc, vc, ks, vs,
                                        mc, status, None)


def _decode(p, q=OK, kc=OK, vc=OK, ks=None, vs=None, mask=OK, lens=OK, tree=None, o=OK, ws=OK, nb=1 << 40):
    return focus._lib.focus_decode_tree(ctypes.byref(p), q, kc, vc, ks, vs, mask, lens, tree, o, None, ws, nb, None)


BAD = [dict(B=0), dict(cap=0), dict(T=0), dict(H=7), dict(R=3), dict(K=33), dict(top_k=5), dict(w=0), dict(format=3)]


@host_only
def test_cache_argument_errors():
    for bad in BAD:
        assert _write(_cp(**bad)) == E["FOCUS_ERR_INVALID_ARG"], bad
    assert _write(_cp(d_head=96)) == E["FOCUS_ERR_UNSUPPORTED"]
    assert _write(_cp(cap=(1 << 30) + 1)) == _write(_cp(B=1 << 20, cap=1 << 24)) == E["FOCUS_ERR_UNSUPPORTED"]
    for name in ("k", "v", "start", "kc", "vc", "mc"):
        assert _write(_cp(), **{name: None}) == E["FOCUS_ERR_INVALID_ARG"], name
    assert _write(_cp(), ks=OK, vs=OK) == _write(_cp(format=1), ks=OK) == E["FOCUS_ERR_INVALID_ARG"]
    assert _write(_cp(), k=P(4104)) == _write(_cp(), kc=P(4104)) == _write(_cp(), status=P(4098)) == E["FOCUS_ERR_ALIGNMENT"]
    odd = focus._Strides(1000, 260, 128)
    assert _write(_cp(), st=ctypes.byref(odd)) == E["FOCUS_ERR_ALIGNMENT"]
    plan = focus.Rope(dim=128)
    assert _write(_cp(d_head=64), rope=plan._addr) == E["FOCUS_ERR_INVALID_ARG"]

    def read(p, kc=OK, vc=OK, ks=None, vs=None, k=OK, v=OK):
        return focus._lib.focus_cache_read(ctypes.byref(p), kc, vc, ks, vs, None, None, k, v, None, None)
    assert read(_cp(), k=None) == read(_cp(), kc=None) == read(_cp(format=2)) == E["FOCUS_ERR_INVALID_ARG"]
    assert read(_cp(), v=P(4100)) == E["FOCUS_ERR_ALIGNMENT"]
    for bad in BAD:
        assert read(_cp(**bad)) == E["FOCUS_ERR_INVALID_ARG"], bad


@host_only
def test_decode_tree_argument_errors():
    for bad in BAD:
        assert _decode(_cp(**bad)) == E["FOCUS_ERR_INVALID_ARG"], bad
        assert focus._lib.focus_decode_tree_workspace_size(ctypes.byref(_cp(**bad))) == 0
    assert _decode(_cp(T=65, cap=100)) == _decode(_cp(H=8192, H_kv=2)) == _decode(_cp(B=65536)) == E["FOCUS_ERR_UNSUPPORTED"]
    assert _decode(_cp(T=10, cap=9)) == E["FOCUS_ERR_INVALID_ARG"]
    for name in ("q", "kc", "vc", "mask", "lens", "o", "ws"):
        assert _decode(_cp(), **{name: None}) == E["FOCUS_ERR_INVALID_ARG"], name
    assert _decode(_cp(), ks=OK, vs=OK) == _decode(_cp(format=2)) == E["FOCUS_ERR_INVALID_ARG"]
    assert _decode(_cp(), tree=P(4100)) == _decode(_cp(), q=P(4104)) == _decode(_cp(), ws=P(4096 + 128)) == E["FOCUS_ERR_ALIGNMENT"]
    need = focus._lib.focus_decode_tree_workspace_size(ctypes.byref(_cp()))
    assert need > 0 and _decode(_cp(), nb=need - 1) == E["FOCUS_ERR_WORKSPACE"]


def test_binding_refuses_wrong_tensors_on_the_host():
    """CPU tensors, wrong shapes and types never reach the library."""
    p = focus.CacheParams(B=1, cap=8, H=2, H_kv=1, d_head=64, R=1, K=2, top_k=1, w=4, format="int8")
    c = focus.KVCache.empty(p, device="cpu")
    assert c.k.dtype == torch.int8 and c.k_scale.shape == (1, 1, 8) and c.mask.shape == (1, 1, 8)
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(focus.FocusError):
        focus.cache_write(p, c, x, x, None, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(focus.FocusError):
        focus.cache_read(p, c, 2)
    with pytest.raises(focus.FocusError):
        focus.decode_tree(p, torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), c, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(focus.FocusError):
        focus.rope(focus.Rope(dim=64), x)
    with pytest.raises(focus.FocusError):
        focus.KVCache.empty(focus.CacheParams(1, 8, 2, 1, 64, 1, 2, 1, 4, "int4"), device="cpu")


def test_reference_pins():
    """The 64-bit definitions themselves: a window over everything and one group are dense
    causal attention; a rotation turns back."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(1, n, 2, 64, generator=g).double() for n in (3, 10, 10))
    mask = torch.ones(1, 1, 10, dtype=torch.int32)
    chain = [[1, 3, 7]]
    for w, m in ((1 << 30, 0 * mask), (1, mask)):
        o, lse, _, _, _ = ref.decode_tree(q, k, v, m, [7], chain, w=w, R=1)
        bias = torch.full((3, 10), -math.inf, dtype=torch.float64).triu(8)
        want = torch.nn.functional.scaled_dot_product_attention(
            q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), attn_mask=bias).transpose(1, 2)
        assert (o - want).abs().max() <= 1e-12
    x = torch.randn(2, 5, 3, 64, generator=g)
    pos = torch.arange(5).expand(2, 5) * 1000
    for layout in ("half", "interleaved"):
        y, _ = ref.rotate(x, pos, 48, layout)
        z, _ = ref.rotate(y, pos, 48, layout, inverse=True)
        assert (z - x.double()).abs().max() <= 1e-12 and (y - x.double()).abs().max() > 1


@host_only
def test_overlaps_are_refused():
    """Outputs that share memory with what is still read, or with themselves."""
    bad = E["FOCUS_ERR_INVALID_ARG"]
    at = lambda i: P((1 << 12) + (i << 24))
    size = 2 * 64 * 2 * 128 * 2  # the cache's bytes
    free = dict(k=at(1), v=at(2), kc=at(3), vc=at(4), mc=at(5), mask=at(6), start=at(7))
    assert _write(_cp(), **{**free, "vc": free["kc"]}) == bad
    for x in ("k", "v"):
        for y in ("kc", "vc"):
            last = P(free[y].value + size - 256)
            assert _write(_cp(), **{**free, x: free[y]}) == _write(_cp(), **{**free, x: last}) == bad, (x, y)

    def read(kc, vc, k, v):
        return focus._lib.focus_cache_read(ctypes.byref(_cp()), kc, vc, None, None, None, None, k, v, None, None)
    assert read(at(1), at(2), at(3), at(3)) == read(at(1), at(2), at(1), at(3)) == read(at(1), at(2), at(3), at(2)) == bad
    assert _decode(_cp(), q=at(1), o=at(1), kc=at(2), vc=at(3)) == bad
    assert _decode(_cp(), q=at(1), o=P(at(1).value + 256), kc=at(2), vc=at(3)) == bad
    plan = focus.Rope(dim=64)._plan
    for st in ((0, 256, 128), (1024, 0, 128), (1024, 256, 0)):
        rc = focus._lib.focus_rope_apply(ctypes.addressof(plan), 0, 2, 4, 2, 0, 128, at(1), None, None, None, None, 0, 0,
                                         at(2), ctypes.byref(focus._Strides(*st)), None, None, None)
        assert rc == bad, st
