"""The ends of the range of the serving operators: scales far apart, roundings counted one by
one, codes at ties, keys that are not finite in long sequences.

References are 64-bit, on the device for long sequences.  Where all cached keys lie in the
window and the drafted tokens form a chain, attention is causal attention: `dense`.
u(t) = eps(t) / 2 is the largest relative error of one rounding to type t.
"""
import math
import threading

import pytest
import torch

import serving_ref as ref

focus = pytest.importorskip("learned_centroid_gated_gb300")

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def u(dtype):
    return torch.finfo(dtype).eps / 2


def randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def dense(p, c, q, lens):
    """o [B, T, H, d], lse [B, H, T], m = sum_j p_j |v_j| and z = max_j (p_j vs_j) sum_j |code_j|
    in 64 bits, every key of the chain seen."""
    B, T, H, d = q.shape
    gq = H // p.H_kv
    o, m, z = (torch.zeros(B, T, H, d, dtype=torch.float64, device="cuda") for _ in range(3))
    lse = torch.zeros(B, H, T, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b] + T
        see = torch.arange(n, device="cuda")[None] <= lens[b] + torch.arange(T, device="cuda")[:, None]
        for g in range(p.H_kv):
            k, v = c.k[b, :n, g].double(), c.v[b, :n, g].double()
            vs = None
            if c.k_scale is not None:
                k = k * c.k_scale[b, g, :n, None].double()
                vs = c.v_scale[b, g, :n].double()
            code, v = v, v if vs is None else v * vs[:, None]
            for h in range(g * gq, (g + 1) * gq):
                s = (q[b, :, h].cuda().double() @ k.T) * p.scale
                s = s.masked_fill(~see, -math.inf)
                top = s.amax(1)
                lse[b, h] = top + (s - top[:, None]).exp().sum(1).log()
                w = (s - lse[b, h][:, None]).exp()
                o[b, :, h], m[b, :, h] = w @ v, w @ v.abs()
                if vs is not None:
                    z[b, :, h] = (w * vs).amax(1)[:, None] * (see.double() @ code.abs())
    return o, lse, m, z


# rows per KV head of the four forms of the kernels: one warp with 8 and with 16 rows, tensor
# cores with up to 128 and up to 256 rows (a capacity of 8000 slots makes them worth it)
FORMS = {"rows_8": 1, "rows_16": 4, "rows_128": 16, "rows_256": 64}


def codes_cache(fmt, B=2, cap=8000, seed=0, **kw):
    p = focus.CacheParams(B=B, cap=cap, **{**dict(H=16, H_kv=4, d_head=128, R=1, K=1, top_k=1, w=1 << 30), **kw}, format=fmt)
    c = focus.KVCache.empty(p)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k, c.v):
        x = torch.randn(t.shape, generator=g, device="cuda")
        t.copy_((x * 40).clamp(-127, 127).round().to(torch.int8) if fmt == "int8" else (x * 140).clamp(-448, 448).to(t.dtype))
    unit = 40.0 if fmt == "int8" else 140.0
    for t in (c.k_scale, c.v_scale):
        t.copy_((torch.rand(t.shape, generator=g, device="cuda") + 0.5) / unit)
    c.mask.fill_(1)
    return p, c


def plain_cache():
    p = focus.CacheParams(B=2, cap=8000, H=16, H_kv=4, d_head=128, R=1, K=1, top_k=1, w=1 << 30)
    c = focus.KVCache.empty(p)
    g = torch.Generator(device="cuda").manual_seed(4)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    c.mask.fill_(1)
    return p, c


# log2 of V's scale by key: None is a scale of zero
SPREADS = {
    "zeros_then_large": lambda j, n: torch.where(j < n // 2, -math.inf, 50.0),
    "large_then_zeros": lambda j, n: torch.where(j < n // 2, 50.0, -math.inf),
    "smallest_to_largest": lambda j, n: -105.0 + 215.0 * j / n,
    "largest_to_smallest": lambda j, n: 110.0 - 215.0 * j / n,
    "blocks": lambda j, n: torch.tensor([-60.0, 100.0, -math.inf, 0.0, -100.0])[(j // 64) % 5],
    "mixed": lambda j, n: torch.tensor([-60.0, 100.0, -math.inf, 0.0, -100.0])[(j * 7) % 5],
}


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("form", FORMS)
def test_scales_at_the_ends_of_the_range(form, spread, fmt):
    """V's scales from 2^-105 to 2^110 and zeros, in tiles of one segment and in different
    segments: a key counts in the sum of the exponentials whatever its V row's size.  The sum of
    the exponentials is checked by LSE, to the bound that holds for scales alike."""
    T, lens = FORMS[form], [2990, 700]
    p, c = codes_cache(fmt)
    n = max(lens) + T
    j = torch.arange(n)
    c.v_scale[:, :, :n] *= torch.exp2(SPREADS[spread](j, n).double()).float().cuda()
    for equal in (True, False):
        if equal:
            keep = c.k_scale.clone()
            c.k_scale.zero_()  # equal logits
        q = randn(p.B, T, p.H, p.d_head, seed=3)
        o, lse = focus.decode_tree(p, q.cuda(), c, torch.tensor(lens, **I32))
        want, want_lse, m, z = dense(p, c, q, lens)
        if equal:
            c.k_scale.copy_(keep)
        # the logits' own error: d 2^-22 of a product of magnitudes below 100
        ds = 0.0 if equal else p.d_head * 2.0 ** -22 * 100
        assert float((lse.double() - want_lse).abs().max()) <= 2 * ds + 2.0 ** -18 * float(want_lse.abs().max())
        # as for scales alike; an output below fp32's normal numbers may be zero
        bound = (u(torch.float16) + 4 * ds + 2.0 ** -18) * m + u(torch.bfloat16) * want.abs() + 2.0 ** -28 * z + 2.0 ** -126
        err = (o.double() - want).abs()
        assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("form", FORMS)
def test_weights_of_8_bit_rows_are_rounded_once(form, fmt):
    """One key with a value among keys whose values are zero, weights from the query: the result
    before its own rounding is off by the one rounding of its weight times its scale to fp16,
    u(fp16), and by 2^-18 of the exponentials and the sum, no more."""
    T = FORMS[form]
    p, c = codes_cache(fmt, H=32, H_kv=8, softmax_scale=1.0)
    lens = [40, 40]
    c.v_scale.zero_(), c.k_scale.zero_()
    g = torch.Generator().manual_seed(9)
    code = torch.randint(1, 127, (p.B, p.H_kv, p.d_head), generator=g).float() * (1 if fmt == "int8" else 3.5)
    c.k[:, 11] = torch.zeros(()).to(c.k.dtype).cuda()
    c.k[:, 11, :, 0] = torch.ones(()).to(c.k.dtype).cuda()
    c.v[:, 11] = code.to(c.v.dtype).cuda()
    c.k_scale[:, :, 11] = 1.0
    c.v_scale[:, :, 11] = 1 + torch.rand(p.B, p.H_kv, generator=g).cuda()
    q = torch.zeros(p.B, T, p.H, p.d_head)
    q[..., 0] = -4 * torch.rand(p.B, T, p.H, generator=g)
    q = q.to(torch.bfloat16)
    o, lse = focus.decode_tree(p, q.cuda(), c, torch.tensor(lens, **I32))
    want, want_lse, _, _ = dense(p, c, q, lens)
    off = (u(torch.float16) + 2.0 ** -18) * want.abs()
    ulp = torch.exp2(torch.floor(torch.log2(want.abs() + off))) * 2.0 ** -7
    err = (o.double() - want).abs() - ulp / 2
    assert bool((err <= off).all()), float((err / want.abs()).max() * 2 ** 11)
    assert float((lse.double() - want_lse).abs().max()) <= 2.0 ** -18 * 8


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H_kv", [1, 16])
def test_codes_at_ties(fmt, H_kv):
    """Codes are round(x (M / max|x|)), ties to even, equal to the last code: rows whose largest
    value divides M exactly and others, filled with values half-way between codes.  The quotient is
    an fp32 number; its product with x is one too for e4m3, and exact for int8, where the code is
    rounded from a fused multiply-add (8 by 24 bits: exact in 64-bit arithmetic here)."""
    M = ref.MAX_CODE[fmt]
    tops = [2.0 ** e * (7 if fmt == "e4m3" else 127) / 64 for e in range(-20, 20)] + [float(x) for x in range(1, 256)]
    g = torch.Generator().manual_seed(2)
    rows = []
    for i, top in enumerate(tops):
        code = torch.randint(0, 127, (4, 128), generator=g).float() + 0.5 if fmt == "int8" else \
            torch.exp2(torch.randint(-5, 8, (4, 128), generator=g).float()) * (2 * torch.randint(8, 16, (4, 128), generator=g) + 1) / 16
        x = (code * (top / M)).clamp(max=top) * (1 - 2 * torch.randint(0, 2, (4, 128), generator=g))
        x[:, 5] = top
        rows.append(x)
    x = torch.cat(rows).to(torch.bfloat16)
    T = len(x) // H_kv
    x = x[:T * H_kv].view(1, T, H_kv, 128)
    p = focus.CacheParams(B=1, cap=T, H=H_kv, H_kv=H_kv, d_head=128, R=1, K=1, top_k=1, w=1, format=fmt)
    c = focus.KVCache.empty(p)
    focus.cache_write(p, c, x.cuda(), x.cuda(), None, torch.zeros(1, **I32))
    f = x.float()
    top = f.abs().amax(-1, keepdim=True)
    y = (f.double() if fmt == "int8" else f) * (torch.tensor(M) / top)
    want = y.round().to(torch.int8) if fmt == "int8" else y.clamp(-M, M).to(torch.float8_e4m3fn)
    for got in (c.k, c.v):
        bad = got.cpu().view(torch.uint8) != want.view(torch.uint8)
        assert int(bad.sum()) == 0, (int(bad.sum()), bad.numel())


def _time(call, n=3):
    call()
    best = math.inf
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("T,H_kv,places", [(1, 8, 1), (1, 1, 2), (16, 8, 1), (16, 8, 3), (64, 8, 1)])
def test_keys_that_are_not_finite_in_a_long_sequence(fmt, T, H_kv, places):
    """V rows of NaN among 100000 keys that half of the tokens see: the rows that see them are
    NaN, the others keep their values, and the call stays of the order of a call without them
    (what is worked out again is their parts of the sequence)."""
    n, at = 100000, [61234, 100, 99990][:places]
    p = focus.CacheParams(B=1, cap=n + 64, H=32, H_kv=H_kv, d_head=128, R=1, K=2, top_k=1, w=4, format=fmt)
    g = torch.Generator(device="cuda").manual_seed(1)
    c = focus.KVCache.empty(p)
    if fmt == "bf16":
        c.k.copy_(torch.randn(c.k.shape, generator=g, device="cuda") * 0.3), c.v.copy_(torch.randn(c.v.shape, generator=g, device="cuda"))
    else:
        for t in (c.k, c.v):
            t.copy_(torch.randint(-127, 128, t.shape, generator=g, device="cuda"))
        c.k_scale.fill_(0.004), c.v_scale.fill_(0.02)
    c.mask.copy_(torch.randint(1, 3, c.mask.shape, generator=g, device="cuda"))
    c.mask[:, :, n:] = 1
    if T > 1:
        c.mask[:, :, n + T // 2:] = 2
    c.mask[0, 0, at] = 1
    q = randn(1, T, p.H, p.d_head, seed=2).cuda()
    lens = torch.tensor([n], **I32)
    ws = torch.empty(focus.decode_tree_workspace_size(p, T), dtype=torch.uint8, device="cuda")
    call = lambda: focus.decode_tree(p, q, c, lens, ws=ws)
    clean, clean_lse = call()
    plain = _time(call)
    if fmt == "bf16":
        c.v[0, at, :, ::2] = math.nan
    else:
        c.v_scale[0, :, at] = math.nan
    got, lse = call()
    hit = _time(call)
    sees = slice(0, max(1, T // 2))
    cols = slice(0, None, 2 if fmt == "bf16" else 1)
    assert bool(got[0, sees, :, cols].isnan().all())
    if fmt == "bf16":  # a column without a NaN keeps its value: 100000 terms in fp32
        err = (got[0, sees, :, 1::2].float() - clean[0, sees, :, 1::2].float()).abs()
        assert bool((err <= 2.0 ** -7 * clean[0, sees, :, 1::2].float().abs() + 2.0 ** -12).all()), float(err.max())
    if T > 1:
        rest = slice(T // 2, None)
        err = (got[0, rest].float() - clean[0, rest].float()).abs()
        assert bool((err <= 2.0 ** -7 * clean[0, rest].float().abs() + 2.0 ** -12).all()), float(err.max())
        assert bool(lse[0, :, rest].isfinite().all())
    print("a clean call %.3f ms, with the key %.3f ms" % (plain, hit))
    assert hit <= 20 * plain + 1.0


def test_a_decode_that_times_out_leaves_nan_and_a_usable_context():
    """The tensor-core kernel with one arrival kept back: its waits run out, every role gives up,
    and the rows are NaN rather than what stood in the workspace.  The next call is right."""
    for _ in range(2):
        assert focus.ERRORS[focus.selftest_timeout_decode()] == "FOCUS_ERR_TIMEOUT"
    for fmt in ("bf16", "int8"):
        for T in (16, 64):
            p, c = (codes_cache(fmt) if fmt != "bf16" else plain_cache())
            lens = [700, 31]
            q = randn(p.B, T, p.H, p.d_head, seed=5)
            ws = torch.empty(focus.decode_tree_workspace_size(p, T), dtype=torch.uint8, device="cuda")
            o, lse = focus.decode_tree(p, q.cuda(), c, torch.tensor(lens, **I32), ws=ws)
            assert focus.get_status(ws) == 0
            want, want_lse, m, _ = dense(p, c, q, lens)
            # one rounding of P, one of the result; logits of magnitudes below 100 off by d 2^-22 of them
            ds = p.d_head * 2.0 ** -22 * 100
            bound = (u(torch.bfloat16) + 4 * ds + 2.0 ** -18) * m + u(torch.bfloat16) * want.abs()
            assert bool(((o.double() - want).abs() <= bound).all())
            assert float((lse.double() - want_lse).abs().max()) <= 2 * ds + 2.0 ** -18 * 16


def test_a_status_word_outlives_the_workspace():
    """A decode without a workspace of the caller's: its code, and that of a captured one, is in
    the status word, which keeps it; a call that fits leaves it alone."""
    p, c = plain_cache()
    q = randn(p.B, 2, p.H, p.d_head, seed=5).cuda()
    good, bad = torch.tensor([5, 7], **I32), torch.tensor([5, p.cap - 1], **I32)
    status = torch.zeros(1, **I32)
    want = focus.decode_tree(p, q, c, good)[0]
    assert torch.equal(focus.decode_tree(p, q, c, good, status=status)[0], want) and focus.get_status(status) == 0
    focus.decode_tree(p, q, c, bad, status=status)
    focus.decode_tree(p, q, c, good, status=status)
    assert focus.ERRORS[focus.get_status(status)] == "FOCUS_ERR_BOUNDS"
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    status.zero_()
    side.wait_stream(torch.cuda.current_stream())
    focus.decode_tree(p, q, c, bad, status=status, stream=side)
    assert focus.ERRORS[focus.get_status(status, side)] == "FOCUS_ERR_BOUNDS"
    torch.cuda.current_stream().wait_stream(side)
    status.zero_()
    lens = good.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        focus.decode_tree(p, q, c, lens, status=status)
    graph.replay()
    assert focus.get_status(status) == 0
    lens.copy_(bad)
    graph.replay()
    assert focus.ERRORS[focus.get_status(status)] == "FOCUS_ERR_BOUNDS"
    for wrong in (torch.zeros(2, **I32), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(focus.FocusError):
            focus.decode_tree(p, q, c, good, status=wrong)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("form", FORMS)
def test_large_queries_beside_a_key_that_is_not_finite(form, fmt):
    """Queries near the largest bf16 number, against key scales that bring the logits back, and a
    key of NaN that half of the tokens (of a single one's: none) see: the others keep their values."""
    T, lens = FORMS[form], [600, 77]
    for e in (126, -127):
        half = 2.0 ** (-60 if e > 0 else 60)
        p, c = codes_cache(fmt, K=2, w=4, softmax_scale=2.0 ** -e / half / math.sqrt(128))
        c.k_scale.mul_(half)
        q = (randn(p.B, T, p.H, p.d_head, seed=3).double().clamp(-3.9, 3.9) * 2.0 ** e).to(torch.bfloat16).cuda()
        rest = slice(T // 2, None)
        for b, n in enumerate(lens):
            c.mask[b, :, n:n + T] = 1
            c.mask[b, :, n + T // 2:n + T] = 2
            c.mask[b, :, :n] = 3
            c.mask[b, :, 20] = 1
        n = torch.tensor(lens, **I32)
        clean, clean_lse = focus.decode_tree(p, q, c, n)
        c.v_scale[:, :, 20] = math.nan
        got, lse = focus.decode_tree(p, q, c, n)
        # both within their bound of the truth: m is at most the largest value, logits below 100
        ds = p.d_head * 2.0 ** -22 * 100
        top = float((c.v.float().abs().amax() * c.v_scale.nan_to_num().amax()))
        bound = 2 * (u(torch.float16) + 4 * ds + 2.0 ** -18) * top + 2 * u(torch.bfloat16) * clean[:, rest].float().abs()
        assert bool(((got[:, rest].float() - clean[:, rest].float()).abs() <= bound).all())
        assert float((lse[..., rest] - clean_lse[..., rest]).abs().max()) <= 4 * ds
        if T > 1:
            assert bool(got[:, :T // 2].isnan().all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_cosines_and_sines_to_fp32(layout):
    """Unit vectors in fp32 turn into the cosines and sines themselves.  They are within 2
    steps of their angle's; the angle, taken from the nearest quarter of a turn, is rounded once (2^-24 of
    its at most an eighth of a turn) and cut off at 2^-32 of a turn.  References by the plan's own
    64-bit fractions, which are exact here."""
    plan = focus.Rope(dim=128, layout=layout, base=5e5)
    N, H = 4096, 3
    g = torch.Generator().manual_seed(6)
    pos = torch.cat([torch.arange(N // 4), torch.randint(-(1 << 31), (1 << 31) - 1, (3 * N // 4,), generator=g)])[None]
    x = torch.zeros(1, N, H, 128)
    ia = torch.arange(64) if layout == "half" else 2 * torch.arange(64)
    ib = ia + (64 if layout == "half" else 1)
    x[..., ia] = 1.0
    turn = torch.tensor([int(t) for t in plan._plan.turn])
    phase = (pos[0].long()[:, None] * turn).double() * 2.0 ** -64  # wraps at 2^64: a turn
    want = torch.cos(2 * math.pi * phase), torch.sin(2 * math.pi * phase)
    off = (4 * phase - (4 * phase).round()).abs() * math.pi / 2  # to the nearest quarter
    for heads in (H, 1):  # a warp per token, and several tokens per warp
        many = 1 if heads == H else 3
        y = focus.rope(plan, x[:, :, :heads].repeat(1, many, 1, 1).contiguous().cuda(), positions=pos.repeat(1, many).to(torch.int32).cuda())
        for at, value, other in ((ia, want[0], want[1]), (ib, want[1], want[0])):
            step = torch.exp2(torch.floor(torch.log2(value.abs().clamp(min=2.0 ** -100)))) * 2.0 ** -23
            bound = 2 * step + other.abs() * (off * 2.0 ** -24 + 2 * math.pi * 2.0 ** -32) + 2.0 ** -50
            err = (y[0, :N, :, :][..., at].double().cpu() - value[:, None]).abs()
            assert bool((err <= bound[:, None]).all()), float((err / bound[:, None]).max())


def test_calls_at_once_on_two_streams():
    """Decodes of all forms and writes to two caches, side by side on two streams from two host
    threads: the same bits as one after another."""
    jobs = []
    for i, (fmt, T) in enumerate([("int8", 1), ("e4m3", 16), ("int8", 64), ("e4m3", 4)]):
        p, c = codes_cache(fmt, seed=i)
        jobs.append((p, c, randn(p.B, T, p.H, p.d_head, seed=i).cuda(), torch.tensor([2000 + 300 * i, 77], **I32),
                     randn(p.B, T, p.H_kv, p.d_head, seed=i + 9).cuda()))
    plan = focus.Rope(dim=128)

    def run(job, stream=None):
        p, c, q, n, k = job
        focus.cache_write(p, c, k, k, None, n, rope=plan, stream=stream)
        return focus.decode_tree(p, focus.rope(plan, q, offset=7, stream=stream), c, n, stream=stream)

    want = [run(job) for job in jobs]
    torch.cuda.synchronize()
    got, failed = [None] * len(jobs), []

    def work(mine):
        try:
            stream = torch.cuda.Stream()
            for _ in range(25):
                for i in mine:
                    got[i] = run(jobs[i], stream)
            stream.synchronize()
        except Exception as e:  # seen by the test below
            failed.append(e)
    threads = [threading.Thread(target=work, args=(m,)) for m in ((0, 1), (2, 3))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed
    for (o, lse), (o2, lse2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
