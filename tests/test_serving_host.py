"""Host side of the serving calls (no GPU needed): plans that are copied, pickled and shared,
tensors that overlap."""
import copy
import ctypes
import decimal
import gc
import multiprocessing
import pickle
import random
import threading
import types

import pytest
import torch

import learned_centroid_gated_gb300 as focus

COPIES = {"copy": copy.copy, "deepcopy": copy.deepcopy,
          "pickle": lambda x: pickle.loads(pickle.dumps(x)),
          "pickle_0": lambda x: pickle.loads(pickle.dumps(x, protocol=0)),
          "inside": lambda x: copy.deepcopy({"layers": [x]})["layers"][0]}


def plan_bytes(rope):
    """The struct that a call through `rope` passes: what stands at its address."""
    own = ctypes.addressof(rope._plan)
    assert rope._addr == own
    return ctypes.string_at(own, ctypes.sizeof(rope._plan))


def cache_bytes(p, T):
    c = p.c(T)
    assert c.addr == ctypes.addressof(c)
    return ctypes.string_at(c.addr, ctypes.sizeof(c))


@pytest.mark.parametrize("how", COPIES)
def test_copies_of_a_plan_pass_their_own_struct(how):
    rope = focus.Rope(dim=96, scaling="by_parts", factor=4.0, layout="interleaved")
    want = plan_bytes(rope)
    other = COPIES[how](rope)
    assert other == rope and hash(other) == hash(rope)
    del rope
    gc.collect()
    noise = [focus.Rope(dim=2) for _ in range(64)]  # takes the memory that was given back
    assert plan_bytes(other) == want and len(noise) == 64
    with pytest.raises(Exception):
        other.dim = 4  # still frozen


@pytest.mark.parametrize("how", COPIES)
def test_copies_of_cache_params_pass_their_own_struct(how):
    p = focus.CacheParams(B=2, cap=100, H=8, H_kv=2, d_head=128, R=1, K=4, top_k=2, w=16, format="e4m3")
    want, ws = [cache_bytes(p, T) for T in (1, 5)], focus.decode_tree_workspace_size(p, 5)
    other = COPIES[how](p)
    assert other == p and hash(other) == hash(p)
    struct = COPIES[how](p.c(5))
    del p
    gc.collect()
    noise = [focus.CacheParams(B=7, cap=7, H=7, H_kv=7, d_head=64, R=1, K=4, top_k=2, w=16).c(1) for _ in range(64)]
    assert [cache_bytes(other, T) for T in (1, 5)] == want and len(noise) == 64
    assert focus.decode_tree_workspace_size(other, 5) == ws
    assert struct.addr == ctypes.addressof(struct)


def _child(data, out):
    rope, p = pickle.loads(data)
    out.put((plan_bytes(rope), cache_bytes(p, 3)))


def test_plans_sent_to_another_process():
    rope = focus.Rope(dim=64)
    p = focus.CacheParams(B=1, cap=64, H=4, H_kv=4, d_head=64, R=1, K=4, top_k=1, w=8)
    want = plan_bytes(rope), cache_bytes(p, 3)
    ctx = multiprocessing.get_context("spawn")
    out = ctx.Queue()
    child = ctx.Process(target=_child, args=(pickle.dumps((rope, p)), out))
    child.start()
    got = out.get(timeout=120)
    child.join(60)
    assert child.exitcode == 0 and got == want


def test_cache_params_shared_by_threads():
    p = focus.CacheParams(B=1, cap=64, H=4, H_kv=4, d_head=64, R=1, K=4, top_k=1, w=8)
    bad = []

    def work():
        for _ in range(50):
            for T in range(1, 33):
                if focus._CacheParams.from_buffer_copy(cache_bytes(p, T)).T != T:
                    bad.append(T)
    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_a_stream_of_another_device_is_refused():
    """Before anything is launched: the tensors' device would not be the current one."""
    other = types.SimpleNamespace(device=torch.device("cuda", 1), device_index=1, cuda_stream=0)
    with pytest.raises(focus.FocusError):
        focus._Launch(0, other)


@pytest.mark.parametrize("call", [focus.rope, focus.rope_bwd])
def test_positions_and_an_offset_together_are_refused(call):
    """One of them would be ignored without a word."""
    x, pos = torch.zeros(1, 2, 1, 64), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(focus.FocusError, match="positions and offset"):
        call(focus.Rope(dim=64), x, positions=pos, offset=3)


# ------------------------------------------------------------------------- frequencies --
D = decimal.Decimal


def two_pi():
    """By Machin's formula, to the context's digits."""
    def atan_of_one_over(n):
        x, total, k = D(1) / n, D(0), 0
        while abs(x) > D(10) ** -(decimal.getcontext().prec + 2):
            total += x / (2 * k + 1) if k % 2 == 0 else -x / (2 * k + 1)
            x, k = x / (n * n), k + 1
        return total
    return 8 * (4 * atan_of_one_over(5) - atan_of_one_over(239))


def turns(dim, base=10000.0, scaling="none", factor=1.0, orig_len=4096, beta_fast=32.0, beta_slow=1.0):
    """f_i / 2 pi to 60 digits, from the definition."""
    pi2, base, factor = two_pi(), D(base), D(factor)
    if scaling == "ntk":
        base *= factor ** (D(dim) / max(dim - 2, 1))
    for i in range(dim // 2):
        f = base ** (D(-2 * i) / dim)
        if scaling == "linear":
            f /= factor
        if scaling == "by_parts":
            keep = min(D(1), max(D(0), (orig_len * f / pi2 - D(beta_slow)) / (D(beta_fast) - D(beta_slow))))
            f = f * (1 - keep) / factor + f * keep
        yield f / pi2


@pytest.mark.parametrize("kw", [dict(dim=128), dict(dim=2), dict(dim=64, base=5e5), dict(dim=126, base=1.0), dict(dim=6, base=1e15),
                                dict(dim=100, scaling="linear", factor=3.0), dict(dim=128, scaling="ntk", factor=8.7),
                                dict(dim=2, scaling="ntk", factor=8.0), dict(dim=4, scaling="ntk", factor=1.1),
                                dict(dim=128, scaling="by_parts", factor=32.0, orig_len=8192),
                                dict(dim=96, scaling="by_parts", factor=3.3, orig_len=777, beta_fast=20.1, beta_slow=0.3)])
def test_frequencies_are_the_nearest_64_bit_fractions(kw):
    """Each f_i / 2 pi in units of 2^-64, so the angle of position p is off by |p| 2^-65 turns at
    most: 2^-34 at the ends of 32 bits.  (Half a unit, and 2^-96 relative of the way there.)"""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        plan = focus.Rope(**kw)._plan
        want = [t * 2 ** 64 for t in turns(**kw)]
        assert len(want) == kw["dim"] // 2
        for got, exact in zip(plan.turn, want):
            assert abs(got - exact) <= D("0.5") + D("0.0001"), (got, exact)
        assert not any(plan.turn[len(want):])


# ------------------------------------------------------------------------- overlaps --
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="passes made-up device addresses; host-only check")
BAD, CUDA = -1, -4  # refused; gone on to the launch, which a machine without a GPU fails
AT = 1 << 20


def rope_call(B, N, d, size, views, positions=None):
    """focus_rope_apply on made-up addresses: views of q, k, q_out, k_out as (address, heads, strides)."""
    plan = focus.Rope(dim=64)
    arg = []
    for v in views:
        arg += [None, None] if v is None else [ctypes.c_void_p(v[0]), ctypes.byref(focus._Strides(*v[2]))]
    return focus._lib.focus_rope_apply(plan._addr, 2 if size == 4 else 0, B, N, views[0][1], views[1][1] if views[1] else 0,
                                       d, *arg[:4], positions, 0, 0, *arg[4:], None)


def elements(B, N, d, size, v):
    return {v[0] + size * (b * v[2][0] + n * v[2][1] + h * v[2][2]) + i
            for b in range(B) for n in range(N) for h in range(v[1]) for i in range(0, d * size, size)}


@host_only
def test_rotation_refuses_outputs_that_overlap():
    """Packed views, shifted views, dense tensors side by side: refused exactly where elements are
    shared, by the elements themselves."""
    rng = random.Random(1)
    d, size, refused, taken = 64, 4, 0, 0
    for _ in range(3000):
        B, N, H, H_kv = rng.choice([1, 2, 3]), rng.choice([1, 2, 5]), rng.choice([1, 2, 4]), rng.choice([1, 2])
        sh = rng.choice([d, d, d + 4, 2 * d])
        heads = rng.choice([H + H_kv, H + H_kv + 3])
        sn = heads * sh + rng.choice([0, 0, 8])
        sb = N * sn + rng.choice([0, 0, sn, 12])
        at = lambda: AT + size * rng.choice([0, 4, sh * rng.randrange(-2, heads + 1), sn * rng.randrange(-1, N + 2) + sh * rng.randrange(0, 3),
                                             sb * rng.randrange(-1, B + 1), rng.randrange(-2 * sn, 2 * sb)])
        q, k = (AT, H, (sb, sn, sh)), (AT + size * H * sh, H_kv, (sb, sn, sh))
        qo = q if rng.random() < 0.3 else (at(), H, (sb, sn, sh))
        ko = k if rng.random() < 0.3 else (at(), H_kv, (sb, sn, sh))
        sets = [elements(B, N, d, size, v) for v in (q, k, qo, ko)]
        meet = lambda i, j: bool(sets[i] & sets[j])
        want = meet(2, 3) or meet(1, 2) or meet(0, 3) or (qo != q and meet(0, 2)) or (ko != k and meet(1, 3))
        got = rope_call(B, N, d, size, (q, k, qo, ko))
        assert got == (BAD if want else CUDA), (B, N, q, k, qo, ko, got, want)
        refused, taken = refused + want, taken + (not want)
    assert refused > 300 and taken > 300
    # dense tensors of different head counts; the positions
    dense = lambda p, H: (p, H, (4 * H * d, H * d, d))
    q, k = dense(AT, 4), dense(AT + (1 << 16), 1)
    assert rope_call(2, 4, d, 4, (q, k, q, k)) == CUDA
    assert rope_call(2, 4, d, 4, (q, k, dense(AT + (1 << 16) - 256, 4), k)) == BAD
    assert rope_call(2, 4, d, 4, (q, k, q, dense(AT + 256 * 31, 1))) == BAD
    assert rope_call(2, 4, d, 4, (q, None, q, None), ctypes.c_void_p(AT + 64)) == BAD
    assert rope_call(2, 4, d, 4, (q, None, q, None), ctypes.c_void_p(AT + 2 * 4 * 4 * d * 4)) == CUDA


@host_only
def test_cache_and_decode_refuse_arrays_that_overlap():
    """Every array that a call writes against every other one, at their first and last bytes."""
    p = focus.CacheParams(B=2, cap=64, H=8, H_kv=2, d_head=128, R=2, K=4, top_k=2, w=16, format="int8").c(3)
    kv, sc, ws = 2 * 64 * 2 * 128, 2 * 2 * 64 * 4, p.tree_ws
    sizes = dict(q=2 * 3 * 8 * 128 * 2, k=2 * 3 * 2 * 128 * 2, v=2 * 3 * 2 * 128 * 2, kc=kv, vc=kv, ks=sc, vs=sc, mc=2 * 2 * 64 * 4,
                 mask=2 * 2 * 3 * 4, n=8, count=8, pos=24, lens=8, tree=48, o=2 * 3 * 8 * 128 * 2, lse=2 * 3 * 8 * 4, ws=ws)
    free = {name: AT + (i << 24) for i, name in enumerate(sizes)}
    P = ctypes.c_void_p

    def write(a):
        return focus._lib.focus_cache_write(p.addr, P(a["k"]), None, P(a["v"]), None, P(a["mask"]), P(a["n"]), P(a["count"]),
                                            None, P(a["pos"]), P(a["kc"]), P(a["vc"]), P(a["ks"]), P(a["vs"]), P(a["mc"]), None, None)

    def read(a):
        return focus._lib.focus_cache_read(p.addr, P(a["kc"]), P(a["vc"]), P(a["ks"]), P(a["vs"]), P(a["n"]), P(a["count"]),
                                           P(a["k"]), P(a["v"]), None, None)

    def decode(a):
        return focus._lib.focus_decode_tree(p.addr, P(a["q"]), P(a["kc"]), P(a["vc"]), P(a["ks"]), P(a["vs"]), P(a["mc"]),
                                            P(a["lens"]), P(a["tree"]), P(a["o"]), P(a["lse"]), P(a["ws"]), ws, None)
    calls = ((write, ("kc", "vc", "ks", "vs", "mc"), ("k", "v", "mask", "n", "count", "pos")),
             (read, ("k", "v"), ("kc", "vc", "ks", "vs", "n", "count")),
             (decode, ("o", "lse", "ws"), ("q", "kc", "vc", "ks", "vs", "mc", "lens", "tree")))
    for call, out, inp in calls:
        assert call(free) == CUDA
        for x in out:
            for y in out + inp:
                if x == y:
                    continue
                last = free[y] + (sizes[y] - 1) // 256 * 256
                assert call({**free, x: free[y]}) == call({**free, x: last}) == BAD, (call.__name__, x, y)
                end = free[y] + (sizes[y] + 255) // 256 * 256
                assert call({**free, x: end}) == CUDA, (call.__name__, x, y)
