"""Acceptance of drafted tokens against a walk of the tree in Python: whole numbers and moved rows,
all of them exact; and the operators of a serving step together."""
import dataclasses
import random

import pytest
import torch

import serving_ref as ref
from test_shared_gpu import I32, filled, masks, params, randn

focus = pytest.importorskip("learned_centroid_gated_gb300")

pytestmark = pytest.mark.gpu


def walk(words, draft, chosen):
    """(path, next) of one sequence."""
    if not words or words[0] != 1:
        return [], -1
    path = [0]
    while True:
        at = path[-1]
        child = [u for u in range(at + 1, len(words)) if words[u] == words[at] | 1 << u and draft[u] == chosen[at]]
        if not child:
            return path, chosen[at]
        path.append(child[0])


def raw(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x


def tensors(c):
    return [x for x in (c.k, c.v, c.k_scale, c.v_scale, c.mask) if x is not None]


def clone(c):
    return focus.KVCache(*[None if x is None else x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale, c.mask)])


def expect(c, lens, paths):
    c = clone(c)
    for b, path in enumerate(paths):
        for i, t in enumerate(path):
            for x in (c.k, c.v):
                raw(x)[b, lens[b] + i] = raw(x)[b, lens[b] + t].clone()
            for x in (c.k_scale, c.v_scale, c.mask):
                if x is not None:
                    x[b, :, lens[b] + i] = x[b, :, lens[b] + t].clone()
    return c


def check(p, c, lens, words, draft, chosen, tree=True):
    tree = torch.tensor(ref.signed(words), dtype=torch.int64, device="cuda") if tree else None
    got = [walk(w, d, x) for w, d, x in zip(words, draft.tolist(), chosen.tolist())]
    want = expect(c, lens, [path for path, _ in got])
    status = torch.zeros(1, **I32)
    n = torch.tensor(lens, **I32)
    count, path, following, new = focus.tree_accept(p, c, n, draft, chosen, tree, status=status)
    T = draft.shape[1]
    assert focus.get_status(status) == 0 and n.tolist() == lens
    assert count.tolist() == [len(x) for x, _ in got]
    assert path.tolist() == [x + [-1] * (T - len(x)) for x, _ in got]
    assert following.tolist() == [x for _, x in got]
    assert new.tolist() == [a + len(x) for a, (x, _) in zip(lens, got)]
    for x, y in zip(tensors(c), tensors(want)):
        assert torch.equal(raw(x), raw(y))
    return got


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("T,tokens", [(1, 2), (2, 1), (5, 2), (33, 2), (64, 1), (64, 2), (64, 3)])
@pytest.mark.parametrize("kw", [dict(), dict(H=3, H_kv=3, d_head=64, R=3), dict(H=40, H_kv=40)])
def test_matches_the_walk(fmt, T, tokens, kw):
    r = random.Random(T * 10 + tokens)
    B = 9
    p = params(B=B, cap=200, format=fmt, **kw)
    c = filled(p, 3)
    lens = [r.randrange(0, 200 - T + 1) for _ in range(B)]
    lens[0], lens[1] = 0, 200 - T
    pick = lambda: torch.tensor([[r.randrange(tokens) for _ in range(T)] for _ in range(B)], **I32)  # noqa: E731
    words = [ref.random_tree(r, T, reach=r.choice([1, 2, 8, 64])) for _ in range(B)]
    words[2] = [0] * T                                  # no token at all
    for t in range(T - T // 3, T):
        words[3][t] = 0                                 # padded
    longest = max(len(x) for x, _ in check(p, c, lens, words, pick(), pick()))
    assert T < 5 or longest > 1
    chain = [[(2 << t) - 1 for t in range(T)]] * B
    check(p, c, lens, chain, pick(), pick(), tree=False)


def test_all_of_a_tree_along_its_last_branch():
    """Every second token on the path: all rows but the root's move, to the sizes of a full draft."""
    T, p = 64, params(B=2, cap=64, H=32, H_kv=32, d_head=128, R=8)
    words = [1] + [(1 | sum(1 << s for s in range(2, t, 2)) | 1 << t) for t in range(1, T)]
    draft = torch.tensor([[t % 2 for t in range(T)]] * 2, **I32)
    chosen = torch.zeros(2, T, **I32)
    got = check(p, filled(p, 5), [0, 0], [words, words], draft, chosen)
    assert got[0][0] == list(range(0, T, 2))


def test_words_that_are_no_tree_and_twins():
    p = params(B=6, cap=40)
    words = [[1, 3, 5, 9], [2, 3, 7, 15], [1, 0b10, 0b101, 0b1111], [0b1001, 0b1011, 0b101, 0b1000], [1, 3, 0b1111, 0b1011],
             [1, 0b11, 0b101, 0b1101]]
    draft = torch.full((6, 4), 7, **I32)
    got = check(p, filled(p, 1), [3, 0, 36, 8, 9, 10], words, draft, torch.full((6, 4), 7, **I32))
    assert [x for x, _ in got] == [[0, 1], [], [0, 2], [], [0, 1, 3], [0, 1]]


@pytest.mark.parametrize("T", [2, 3, 8, 33, 64])
def test_words_at_random(T):
    """Words without their own bit, with later ones', copied from other tokens: none of them is accepted."""
    r = random.Random(T)
    B = 200
    p = params(B=B, cap=T + 9)
    words = [ref.random_tree(r, T, reach=r.choice([1, 2, 64])) for _ in range(B)]
    for w in words:
        for _ in range(r.randrange(4)):
            w[r.randrange(T)] = r.choice([r.getrandbits(T), w[r.randrange(T)], w[r.randrange(T)] | 1 << r.randrange(T), 0])
    pick = lambda: torch.tensor([[r.randrange(2) for _ in range(T)] for _ in range(B)], **I32)  # noqa: E731
    check(p, filled(p, 8), [r.randrange(10) for _ in range(B)], words, pick(), pick())


def test_negative_tokens_are_none():
    """A choice of -1 (of a row of logits without a token) and an empty place of a draft are not a
    match, as the root's choice, along a chain, and beside a twin that has a token."""
    p = params(B=4, cap=40)
    c = filled(p, 6)
    words = [[1, 3, 7, 15], [1, 3, 5, 11], [1, 3, 7, 15], [1, 3, 5, 9]]
    draft = torch.tensor([[5, -1, -1, -1], [5, -1, 7, 8], [5, 6, -1, 9], [5, -7, -7, 2]], **I32)
    chosen = torch.tensor([[-1, -1, -1, -1], [7, 8, -1, 4], [6, -1, 9, 9], [-7, 1, 1, 1]], **I32)
    old, n = clone(c), torch.tensor([3, 0, 9, 36], **I32)
    count, path, following, new = focus.tree_accept(p, c, n, draft, chosen, torch.tensor(words, dtype=torch.int64, device="cuda"))
    assert count.tolist() == [1, 2, 2, 1] and following.tolist() == [-1, -1, -1, -7]
    assert path.tolist() == [[0, -1, -1, -1], [0, 2, -1, -1], [0, 1, -1, -1], [0, -1, -1, -1]]
    assert new.tolist() == [4, 2, 11, 37]
    want = expect(old, [3, 0, 9, 36], [[0], [0, 2], [0, 1], [0]])
    for x, y in zip(tensors(c), tensors(want)):
        assert torch.equal(raw(x), raw(y))
    # a chain whose choices are those of logits without a token
    logits = torch.randn(4, 4, 50, device="cuda")
    logits[0, 1], logits[2, 0, 7] = float("nan"), float("inf")
    chosen, _ = focus.sample(logits, torch.full((4, 4), 0.5, device="cuda"))
    assert chosen[0, 1] == chosen[2, 0] == -1
    draft = torch.cat([torch.zeros(4, 1, **I32), chosen[:, :-1]], 1).contiguous()
    count, _, following, _ = focus.tree_accept(p, c, torch.zeros(4, **I32), draft, chosen)
    assert count.tolist() == [2, 4, 1, 4] and following.tolist() == [-1, int(chosen[1, 3]), -1, int(chosen[3, 3])]


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_lengths_in_place_and_outside(fmt):
    p = params(B=70, cap=50, format=fmt)
    c = filled(p, 2)
    lens = [b % 45 for b in range(70)]
    lens[4], lens[5], lens[69] = -1, 46, 2147483647
    n = torch.tensor(lens, **I32)
    same = torch.zeros(70, 5, **I32)
    status = torch.zeros(1, **I32)
    old = clone(c)
    count, path, following, new = focus.tree_accept(p, c, n, same, same, out_lens=n, status=status)
    assert new is n and focus.get_status(status) == -6
    for b in range(70):
        out = b in (4, 5, 69)
        assert int(count[b]) == (0 if out else 5) and int(following[b]) == (-1 if out else 0)
        assert int(n[b]) == lens[b] + (0 if out else 5)
        assert path[b].tolist() == ([-1] * 5 if out else [0, 1, 2, 3, 4])
    for x, y in zip(tensors(c), tensors(old)):
        assert torch.equal(raw(x), raw(y))


def test_refusals():
    p = params(B=2, cap=40)
    c = filled(p, 2)
    n, x = torch.zeros(2, **I32), torch.zeros(2, 4, **I32)
    for bad in ((n, x, x[:, :3].contiguous()), (n[:1], x, x), (n, x.long(), x), (n, x, x, torch.zeros(2, 4, **I32)),
                (n, torch.zeros(2, 65, **I32), torch.zeros(2, 65, **I32)), (n, x.cpu(), x), (n, x[0], x[0])):
        with pytest.raises(focus.FocusError):
            focus.tree_accept(p, c, *bad)
    for kw in (dict(out_lens=torch.zeros(3, **I32)), dict(status=torch.zeros(2, **I32)), dict(out_lens=x[0, :2])):
        with pytest.raises(focus.FocusError):
            focus.tree_accept(p, c, n, x, x, **kw)


# --------------------------------------------------- the operators together, as in use --
class Model:
    """A toy model in place of one: embeddings, one attention layer's projections, and an output
    matrix, of random weights; the attention is the caller's."""

    def __init__(self, V, H, H_kv, d, K, seed=0):
        g = torch.Generator().manual_seed(seed)
        w = 32
        self.emb = torch.randn(V, w, generator=g).cuda()
        self.wq, self.wk, self.wv = (torch.randn(w, n * d, generator=g).cuda() / 6 for n in (H, H_kv, H_kv))
        self.wo = torch.randn(H * d, V, generator=g).cuda() / 10
        self.groups = masks(seed + 1, K, 1, V).cuda()
        self.shape = (H, H_kv, d)

    def qkv(self, tokens):
        H, H_kv, d = self.shape
        x = self.emb[tokens]
        return [(x @ w).to(torch.bfloat16).view(*tokens.shape, n, d) for w, n in ((self.wq, H), (self.wk, H_kv), (self.wv, H_kv))]

    def logits(self, o):
        return o.float().flatten(2) @ self.wo


def steps(model, p, prefix, P, rope, root, noise, n, tree, r, forced=None):
    """n steps of drafting behind the root (three of four guesses are `forced`'s tokens, where it is
    given; with one token a step all are), writing the drafted keys, attention, sampling with random numbers that
    belong to positions, and acceptance.  Returns each sequence's tokens, and the attention's result at each."""
    B, T, V = p.B, len(tree), model.emb.shape[0]
    words = torch.tensor(ref.signed([tree] * B), dtype=torch.int64, device="cuda")
    deep = [bin(x).count("1") - 1 for x in tree]
    depth = torch.tensor(deep, **I32)
    c = focus.KVCache.empty(p)
    out, seen = [[x] for x in root], [[] for _ in range(B)]
    root, lens = torch.tensor(root, **I32), torch.zeros(B, **I32)
    for _ in range(n):
        draft = [[r.randrange(V) for _ in range(T)] for _ in range(B)]
        for b in range(B):
            for t in range(1, T):
                at = len(out[b]) - 1 + deep[t]
                if forced and at < len(forced[b]) and r.random() < 0.75:
                    draft[b][t] = forced[b][at]
        draft = torch.tensor(draft, **I32)
        draft[:, 0] = root
        positions = (P + lens[:, None] + depth).contiguous()
        q, k, v = model.qkv(draft.long())
        focus.cache_write(p, c, k, v, model.groups[draft.long()][:, None].contiguous(), lens, rope=rope, positions=positions)
        o, _ = focus.decode_shared(p, focus.rope(rope, q, positions=positions), prefix, P, c, lens, words)
        u = noise.gather(1, (lens[:, None] + depth).long()).contiguous()
        chosen, _ = focus.sample(model.logits(o), u, temperature=0.6, top_k=40, top_p=0.95)
        count, path, root, new = focus.tree_accept(p, c, lens, draft, chosen, words, out_lens=lens)
        assert new is lens
        for b in range(B):
            for t in path[b].tolist():
                if t >= 0:
                    seen[b].append(o[b, t])
                    out[b].append(int(chosen[b, t]))
            assert int(root[b]) == out[b][-1] and int(lens[b]) == len(out[b]) - 1
        if T == 1 and forced:
            root = torch.tensor([x[len(y) - 1] for x, y in zip(forced, out)], **I32)
            for x, y in zip(forced, out):
                y[-1] = x[len(y) - 1]
    return out, seen


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_drafting_sampling_and_acceptance_together(fmt):
    """What drafts and acceptance make of a sequence is what its tokens one by one give: the same
    tokens, forced, a step each in a cache of their own, have the same attention results.  Both runs read the
    same K and V (to the code), so that they differ by at most twice a result's bound, in which
    sum p |v| <= max |v|: 2 (u(P) + u(bf16) + 2^-12) max |v|."""
    B, V, P, H, H_kv, d = 3, 50, 300, 8, 2, 64
    model = Model(V, H, H_kv, d, K=4)
    p = params(B=B, cap=200, H=H, H_kv=H_kv, d_head=d, K=4, top_k=1, w=64, format=fmt)
    rope = focus.Rope(dim=d)
    pp = dataclasses.replace(p, B=1, cap=P)
    prefix = focus.KVCache.empty(pp)
    text = torch.randint(0, V, (1, P), generator=torch.Generator().manual_seed(5)).cuda()
    _, k, v = model.qkv(text)
    focus.cache_write(pp, prefix, k, v, model.groups[text][:, None].contiguous(), torch.zeros(1, **I32), rope=rope)
    noise = torch.rand(B, 200, generator=torch.Generator().manual_seed(6)).cuda()
    r = random.Random(7)
    first, _ = steps(model, p, prefix, P, rope, [1, 2, 3], noise, 30, [1], r)
    assert all(len(x) == 31 for x in first)
    tree = [1, 0b11, 0b101, 0b1101, 0b10101, 0b110101]
    got, seen = steps(model, p, prefix, P, rope, [1, 2, 3], noise, 14, tree, r, forced=first)
    assert all(15 < len(x) < 90 for x in got)
    n = min(len(x) for x in got) - 1
    one, plain = steps(model, p, prefix, P, rope, [1, 2, 3], noise, n, [1], r, forced=got)
    assert [x[:n + 1] for x in one] == [x[:n + 1] for x in got]
    most = float(max(model.qkv(torch.arange(V, device="cuda"))[2].abs().max(), v.abs().max()))
    for b in range(B):
        a, c = torch.stack(seen[b][:n]).float(), torch.stack(plain[b][:n]).float()
        assert (a - c).abs().max().item() <= 2 * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -12) * most * 1.07
        assert a.abs().max().item() > 0.1 * most
