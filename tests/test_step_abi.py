"""Host-side checks of sampling, shared-prefix decode and acceptance (no GPU needed): refusals
before anything is launched."""
import ctypes
import math

import pytest
import torch

import learned_centroid_gated_gb300 as focus

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="passes made-up device addresses; host-only check")
E = {v: k for k, v in focus.ERRORS.items()}
P = ctypes.c_void_p


def at(i):
    """Addresses far from one another."""
    return P((i + 1) << 36)


def _sample(logits=at(0), u=at(1), T=None, k=None, p=None, m=None, token=at(2), logprob=at(3), status=None, **kw):
    c = dict(rows=4, V=1000, dtype=0, top_k=0, stride=1000, temperature=1.0, top_p=1.0, min_p=0.0)
    c.update(kw)
    c = focus._SampleParams(*c.values())
    return focus._lib.focus_sample(ctypes.addressof(c), logits, u, T, k, p, m, token, logprob, status, None)


@host_only
def test_sample_argument_errors():
    bad, unsupported, misaligned = (E["FOCUS_ERR_" + x] for x in ("INVALID_ARG", "UNSUPPORTED", "ALIGNMENT"))
    for kw in (dict(logits=None), dict(u=None), dict(token=None), dict(rows=0), dict(V=0), dict(dtype=3), dict(stride=-1),
               dict(temperature=-0.5), dict(temperature=math.nan), dict(temperature=math.inf), dict(top_p=-1.0),
               dict(top_p=math.nan), dict(min_p=-0.1), dict(min_p=1.1), dict(min_p=math.nan)):
        assert _sample(**kw) == bad, kw
    for kw in (dict(V=(1 << 19) + 1), dict(rows=(1 << 24) + 1), dict(stride=1 << 33)):
        assert _sample(**kw) == unsupported, kw
    for kw in (dict(logits=P((1 << 36) + 1)), dict(dtype=2, logits=P((1 << 36) + 2)), dict(u=P((2 << 36) + 2)),
               dict(token=P((3 << 36) + 1)), dict(k=P(4098)), dict(status=P(4097))):
        assert _sample(**kw) == misaligned, kw
    # outputs over inputs, over one another
    for kw in (dict(token=at(1)), dict(logprob=at(2)), dict(logprob=P((1 << 36) + 7996)), dict(T=at(3)), dict(status=at(2))):
        assert _sample(**kw) == bad, kw


def _cp(**kw):
    base = dict(B=2, cap=64, T=3, H=8, H_kv=2, d_head=128, R=1, K=4, top_k=2, w=16, format=0, softmax_scale=0.0)
    base.update(kw)
    return focus._CacheParams(*base.values())


def _shared(p, q=at(0), cap=100, n=50, pk=at(1), pv=at(2), pks=None, pvs=None, pm=at(3), kc=at(4), vc=at(5), ks=None, vs=None,
            mask=at(6), lens=at(7), tree=None, o=at(8), lse=at(9), ws=at(10), nb=1 << 34):
    return focus._lib.focus_decode_shared(ctypes.byref(p), q, cap, n, pk, pv, pks, pvs, pm, kc, vc, ks, vs, mask, lens, tree, o,
                                          lse, ws, nb, None)


@host_only
def test_shared_argument_errors():
    bad, unsupported, misaligned, small = (E["FOCUS_ERR_" + x] for x in ("INVALID_ARG", "UNSUPPORTED", "ALIGNMENT", "WORKSPACE"))
    for kw in (dict(B=0), dict(cap=0), dict(T=0), dict(H=7), dict(R=3), dict(K=33), dict(top_k=5), dict(w=0), dict(format=3)):
        assert _shared(_cp(**kw)) == bad, kw
    for kw in (dict(d_head=96), dict(T=65, cap=100), dict(B=65536)):
        assert _shared(_cp(**kw)) == unsupported, kw
    for kw in (dict(q=None), dict(pk=None), dict(pv=None), dict(pm=None), dict(kc=None), dict(vc=None), dict(mask=None),
               dict(lens=None), dict(o=None), dict(ws=None), dict(cap=0), dict(n=-1), dict(n=101), dict(pks=at(11), pvs=at(12)),
               dict(ks=at(11), vs=at(12))):
        assert _shared(_cp(), **kw) == bad, kw
    eight = dict(pks=at(11), pvs=at(12), ks=at(13), vs=at(14))
    for x in eight:
        assert _shared(_cp(format=1), **{**eight, x: None}) == bad, x
    assert _shared(_cp(cap=1 << 30), cap=1 << 30, n=1 << 30) == unsupported
    assert _shared(_cp(), cap=(1 << 30) + 1) == unsupported
    for kw in (dict(q=P((1 << 36) + 8)), dict(pk=P((2 << 36) + 8)), dict(pm=P((4 << 36) + 2)), dict(tree=P(4100)), dict(ws=P((11 << 36) + 64)),
               dict(o=P((9 << 36) + 2))):
        assert _shared(_cp(), **kw) == misaligned, kw
    assert _shared(_cp(), nb=1000) == small
    for kw in (dict(o=at(0)), dict(o=at(2)), dict(lse=at(3)), dict(ws=at(1)), dict(ws=at(7)), dict(lse=at(8))):
        assert _shared(_cp(), **kw) == bad, kw
    size = focus._lib.focus_decode_shared_workspace_size
    assert size(ctypes.byref(_cp(T=65, cap=100)), 5) == size(ctypes.byref(_cp()), -1) == 0
    assert size(ctypes.byref(_cp()), 50) > focus._lib.focus_decode_tree_workspace_size(ctypes.byref(_cp()))


@host_only
def test_selftest_argument_errors():
    selftest = focus._lib.focus_selftest_timeout_shared
    for ws, size, want in ((None, 1 << 24, "INVALID_ARG"), (P((1 << 36) + 64), 1 << 24, "ALIGNMENT"), (at(0), (1 << 24) - 1, "WORKSPACE")):
        assert selftest(ws, size, None) == E["FOCUS_ERR_" + want]


def _accept(p, draft=at(0), chosen=at(1), tree=None, kc=at(2), vc=at(3), ks=None, vs=None, mc=at(4), lens=at(5), lens_out=at(6),
            count=at(7), path=at(8), following=at(9), status=None):
    return focus._lib.focus_tree_accept(ctypes.byref(p), draft, chosen, tree, kc, vc, ks, vs, mc, lens, lens_out, count, path,
                                        following, status, None)


@host_only
def test_accept_argument_errors():
    bad, unsupported, misaligned = (E["FOCUS_ERR_" + x] for x in ("INVALID_ARG", "UNSUPPORTED", "ALIGNMENT"))
    for kw in (dict(B=0), dict(cap=2), dict(T=0), dict(H=7), dict(R=3), dict(format=3)):
        assert _accept(_cp(**kw)) == bad, kw
    for kw in (dict(d_head=96), dict(T=65, cap=100), dict(B=65536)):
        assert _accept(_cp(**kw)) == unsupported, kw
    for x in ("draft", "chosen", "kc", "vc", "mc", "lens", "lens_out", "count", "path", "following"):
        assert _accept(_cp(), **{x: None}) == bad, x
    assert _accept(_cp(), ks=at(10), vs=at(11)) == _accept(_cp(format=2), ks=at(10)) == bad
    for kw in (dict(draft=P(4098)), dict(tree=P(4100)), dict(kc=P((3 << 36) + 8)), dict(path=P(4097)), dict(status=P(4099))):
        assert _accept(_cp(), **kw) == misaligned, kw
    for kw in (dict(kc=at(3)), dict(count=at(0)), dict(path=at(7)), dict(lens_out=P((6 << 36) + 4)), dict(mc=at(5)),
               dict(status=at(9)), dict(tree=at(8))):
        assert _accept(_cp(), **kw) == bad, kw
