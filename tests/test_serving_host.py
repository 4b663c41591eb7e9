"""Host side of the serving calls (no GPU needed): plans that are copied, pickled and shared."""
import copy
import ctypes
import gc
import multiprocessing
import pickle
import threading

import pytest

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
