"""tgdn_paged_tree_attention against attention in 64 bits: page sizes, head layouts, both
types, trees of 1 to 256 nodes, contexts from nothing to many tiles, whole and split items;
non-finite values in masked places and stale page positions; bad pages and lengths; agreement
with tgdn_tree_attention on a dense cache."""
import numpy as np
import pytest

from tree_speculative_decoding_gated_gb300 import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from attn_helpers import assert_within, attend, visible_tree  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402

BF, HF = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, parents, lens, H_q, H_kv, d, ps, dtype, seed=0, n_max=None, spare=3):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.parents, self.lens, self.ps = [np.asarray(p, np.int32) for p in parents], lens, ps
        n = [len(p) for p in self.parents]
        self.cu = np.r_[0, np.cumsum(n)].astype(np.int32)
        B, T = len(n), int(self.cu[-1])
        randn = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
        self.qkv = randn(T, H_q + 2 * H_kv, d)
        self.q, self.k, self.v = (self.qkv[:, :H_q], self.qkv[:, H_q:H_q + H_kv],
                                  self.qkv[:, H_q + H_kv:])
        held = [-(-x // ps) for x in lens]
        n_pages = sum(held) + spare
        self.pages = tgdn.Pages(B, n_pages, ps, max(held + [1]) + 1)
        ids = rng.permutation(n_pages)
        at = 0
        self.pages.table.fill_(-7)   # never read past the held pages
        for b in range(B):
            self.pages.table[b, :held[b]] = ints(ids[at:at + held[b]])
            at += held[b]
        self.pages.len.copy_(ints(lens))
        self.pages.held.copy_(ints(held))
        self.kp, self.vp = randn(n_pages, H_kv, ps, d), randn(n_pages, H_kv, ps, d)
        for b in range(B):           # stale positions of the last pages, and free pages
            if lens[b] % ps:
                last = int(self.pages.table[b, held[b] - 1])
                self.kp[last, :, lens[b] % ps:] = float("nan")
                self.vp[last, :, lens[b] % ps:] = float("nan")
        for p in ids[at:]:
            self.kp[p] = float("inf")
            self.vp[p] = float("nan")
        self.tree = tgdn.Tree.from_host(self.cu, np.concatenate(self.parents) if T else np.zeros(0, np.int32),
                                        n_max or max(n + [1]), 64)
        tgdn.tree_prep(self.tree)
        self.scale = d ** -0.5

    def run(self, split=True):
        c = self
        o = torch.full(c.q.shape, float("nan"), dtype=c.q.dtype, device="cuda")
        ws = None
        if split:
            nb = tgdn.paged_tree_attention_workspace_bytes(c.tree, c.pages, c.q.shape[1], c.k.shape[1],
                                                           c.q.shape[2])
            assert nb > 0
            ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")   # stale bytes
        tgdn.paged_tree_attention(c.tree, c.pages, c.q, c.k, c.v, c.kp, c.vp, o, c.scale, ws=ws)
        torch.cuda.synchronize()
        return o

    def keys(self, b):
        ids = self.pages.table[b, :-(-self.lens[b] // self.ps)].long()
        cat = lambda pool, new: torch.cat([  # noqa: E731
            pool[ids].transpose(1, 2).reshape(-1, *new.shape[1:])[:self.lens[b]], new])
        s = slice(int(self.cu[b]), int(self.cu[b + 1]))
        return cat(self.kp, self.k[s]), cat(self.vp, self.v[s])

    def check(self, o, skip=()):
        worst = 0.0
        for b, p in enumerate(self.parents):
            if not len(p) or b in skip:
                continue
            s = slice(int(self.cu[b]), int(self.cu[b + 1]))
            k, v = self.keys(b)
            see = np.concatenate([np.ones((len(p), self.lens[b]), bool), visible_tree(p)], 1)
            ref, tol = attend(self.q[s], k, v, see, self.scale)
            worst = max(worst, assert_within(o[s], ref, tol, f"sequence {b}"))
        return worst


def trees(rng, sizes, cap=12):
    return [synth.random_recursive_tree(rng, int(n), cap) if n else np.zeros(0, np.int32)
            for n in sizes]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H_q,H_kv,d", [(4, 1, 128), (6, 2, 64), (3, 3, 96)])
def test_page_sizes_and_ragged_contexts(ps, H_q, H_kv, d, dtype):
    rng = np.random.default_rng(ps + d)
    sizes = [1, 7, 0, 64, 33, 2, 1, 20]
    lens = [0, 1, 50, ps, ps - 1, 127, 129, 700]
    c = Case(trees(rng, sizes), lens, H_q, H_kv, d, ps, dtype, seed=ps)
    for split in (False, True):
        print("share of the tolerance", c.check(c.run(split)))
    assert c.tree.status.tolist() == [0] * 8


@pytest.mark.parametrize("H_q,H_kv,d", [(1, 1, 128), (16, 4, 128), (5, 1, 8), (64, 1, 64), (128, 1, 32),
                                        (7, 1, 112), (16, 16, 64), (33, 1, 128)])
def test_head_layouts(H_q, H_kv, d):
    rng = np.random.default_rng(H_q)
    c = Case(trees(rng, [40, 3, 1]), [300, 15, 40], H_q, H_kv, d, 32, BF, seed=d)
    for split in (False, True):
        c.check(c.run(split))


@pytest.mark.parametrize("G", [1, 4, 8])
def test_trees_up_to_256_nodes(G):
    rng = np.random.default_rng(G)
    parents = trees(rng, [256, 129, 128, 200, 65], 30) + [synth.chain_tree(60)]
    c = Case(parents, [10, 0, 333, 64, 129, 1], 2 * G, 2, 128, 64, BF, seed=G, n_max=256)
    for split in (False, True):
        c.check(c.run(split))


def test_deep_chains_and_relabelled_roots():
    chain = synth.chain_tree(64)                       # 65 nodes, depth 64
    back = np.array([1, 2, 3, -1], np.int32)           # the root is the last node
    star = np.array([2, 2, -1, 2, 2, 2], np.int32)
    c = Case([chain, back, star], [70, 0, 5], 4, 2, 64, 16, BF, seed=3)
    for split in (False, True):
        c.check(c.run(split))


def test_long_context_in_many_parts():
    """One sequence over many tiles: every CTA takes a run, the merge joins dozens of parts."""
    c = Case([np.array([-1], np.int32), np.array([-1, 0, 0], np.int32)], [20000, 3], 2, 1, 64, 64, HF,
             seed=4)
    for split in (False, True):
        c.check(c.run(split))


@pytest.mark.parametrize("nodes,lens,H_q,H_kv,d", [
    ([33, 12, 0, 5], [9000, 6001, 50, 0], 4, 1, 128),      # two row tiles, few items
    ([7, 3], [9500, 5000], 8, 2, 96),                       # 28 rows, joined eight at a time
    ([1, 1, 2], [12000, 1, 7777], 5, 1, 64),                # few rows in all
    ([64] * 9, [1500] * 8 + [900], 16, 4, 128)])            # many items, 32 rows at a time
def test_joins_of_every_kind(nodes, lens, H_q, H_kv, d):
    c = Case(trees(np.random.default_rng(12), nodes), lens, H_q, H_kv, d, 64, BF, seed=13)
    o = c.run(True)
    c.check(o)
    assert torch.equal(o, c.run(True))


def test_many_sequences():
    rng = np.random.default_rng(6)
    B = 70
    c = Case(trees(rng, rng.integers(0, 9, B)), rng.integers(0, 400, B).tolist(), 2, 2, 64, 16, BF,
             seed=6)
    for split in (False, True):
        c.check(c.run(split))


def test_runs_are_equal_bit_for_bit():
    rng = np.random.default_rng(7)
    c = Case(trees(rng, [64, 10, 1, 30]), [900, 2000, 64, 1], 8, 2, 128, 64, BF, seed=7)
    a = c.run()
    for _ in range(5):
        assert torch.equal(a, c.run())


def test_masked_values_reach_no_row():
    """Non-finite keys and values of other branches, stale positions (Case fills them) and other
    sequences: the rows that do not see them keep every bit."""
    parent = np.array([-1, 0, 0, 1, 1, 2, 5], np.int32)
    c = Case([parent, parent], [150, 30], 4, 2, 128, 16, BF, seed=8)
    for split in (False, True):
        clean = c.run(split)
        c.check(clean)
        k, v = c.k.clone(), c.v.clone()
        c.v[2, 0, 9] = float("nan")      # node 2: seen by 2, 5, 6
        c.v[4, 1, 0] = float("inf")      # node 4: by itself
        c.k[5, 0] = float("nan")         # node 5: by 5, 6
        got = c.run(split)
        bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
        assert torch.equal(bits(got[[0, 1, 3]]), bits(clean[[0, 1, 3]]))
        assert torch.equal(bits(got[7:]), bits(clean[7:]))
        assert bool(torch.isnan(got[2, :2, 9]).all()) and bool(torch.isnan(got[5:7, :2]).all())
        keep = [x for x in range(128) if x != 9]
        assert torch.equal(bits(got[2][:, keep]), bits(clean[2][:, keep]))
        assert bool((got[4, 2:, 0] == float("inf")).all())
        assert torch.equal(bits(got[4, :2]), bits(clean[4, :2]))
        c.k.copy_(k), c.v.copy_(v)


def test_non_finite_cached_values_are_seen():
    c = Case([np.array([-1, 0], np.int32)], [140], 2, 1, 64, 64, BF, seed=9)
    page, at = int(c.pages.table[0, 2]), 5          # position 133, inside the last, partial tile
    c.vp[page, 0, at, 3] = float("inf")
    o = c.run()
    assert bool((o[:, :, 3] == float("inf")).all())
    assert bool(torch.isfinite(o[:, :, :3]).all())


@pytest.mark.parametrize("split", [False, True])
def test_bad_pages_and_lengths(split):
    rng = np.random.default_rng(10)
    sizes, lens = [5, 6, 7, 8, 9, 4], [300, 900, 40, 128, 77, 300]

    def fresh():
        return Case(trees(np.random.default_rng(10), sizes), lens, 4, 2, 64, 16, BF, seed=10)

    good = fresh().run(split)
    c = fresh()
    c.pages.table[0, 3] = c.pages.n_pages           # just past the pool
    c.pages.table[1, 50] = -1
    c.pages.len[2] = 16 * 3 + 1                       # more than the held pages
    c.pages.held[4] = c.pages.max_pages + 1
    o = c.run(split)
    assert c.tree.status.tolist() == [8, 8, 8, 0, 8, 0]
    for b in (0, 1, 2, 4):
        assert not bool(o[c.cu[b]:c.cu[b + 1]].any()), b
    for b in (3, 5):
        s = slice(int(c.cu[b]), int(c.cu[b + 1]))
        ref = c.check(o, skip=(0, 1, 2, 4))
        assert ref <= 1.0 and bool(torch.isfinite(o[s]).all())
    # the status stays: a later call with mended pages still gives zeros until prep runs again
    c.pages.table[0, 3] = int(fresh().pages.table[0, 3])
    o = c.run(split)
    assert not bool(o[:5].any())
    tgdn.tree_prep(c.tree)
    o = c.run(split)
    assert c.tree.status.tolist()[0] == 0
    s = slice(0, 5)
    assert torch.allclose(o[s].float(), good[s].float(), atol=2.0 ** -6)


def test_invalid_trees_get_zeros():
    bad = [np.array([-1, 0, -1], np.int32), np.array([1, 0], np.int32), np.array([-1, 0], np.int32)]
    c = Case(bad, [40, 200, 40], 4, 2, 64, 16, BF, seed=11)
    for split in (False, True):
        o = c.run(split)
        assert c.tree.status.tolist() == [3, 3, 0]
        assert not bool(o[:5].any())
        c.check(o, skip=(0, 1))


def test_agrees_with_the_dense_cache():
    rng = np.random.default_rng(12)
    lens = [200, 64, 0, 513]
    c = Case(trees(rng, [64, 20, 9, 1]), lens, 16, 4, 128, 64, BF, seed=12)
    P = 520
    kc, vc = torch.zeros(4, P, 4, 128, dtype=BF, device="cuda"), torch.zeros(4, P, 4, 128, dtype=BF,
                                                                             device="cuda")
    for b in range(4):
        k, v = c.keys(b)
        kc[b, :lens[b]], vc[b, :lens[b]] = k[:lens[b]], v[:lens[b]]
    q, k, v = c.q.contiguous(), c.k.contiguous(), c.v.contiguous()
    o = torch.empty_like(q)
    tgdn.tree_attention(c.tree, q, k, v, kc, vc, ints(lens), o, c.scale)
    got = c.run()
    c.check(got)
    for b in range(4):
        s = slice(int(c.cu[b]), int(c.cu[b + 1]))
        kk, vv = c.keys(b)
        see = np.concatenate([np.ones((s.stop - s.start, lens[b]), bool), visible_tree(c.parents[b])], 1)
        _, tol = attend(c.q[s], kk, vv, see, c.scale)
        # each is within its tolerance of the same value
        assert bool(((o[s].cpu().double() - got[s].cpu().double()).abs() <= 2 * tol).all())


def test_no_pages_at_all():
    c = Case([np.array([-1, 0, 1], np.int32)], [0], 4, 2, 64, 16, BF, seed=13, spare=0)
    assert c.pages.n_pages == 0
    for split in (False, True):
        c.check(c.run(split))


def test_in_a_graph_and_on_a_side_stream():
    rng = np.random.default_rng(14)
    c = Case(trees(rng, [64, 1]), [1500, 900], 8, 2, 128, 32, BF, seed=14)
    want = c.run()
    nb = tgdn.paged_tree_attention_workspace_bytes(c.tree, c.pages, 8, 2, 128)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tgdn.paged_tree_attention(c.tree, c.pages, c.q, c.k, c.v, c.kp, c.vp, o, c.scale, ws=ws)
    side.synchronize()
    assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tgdn.paged_tree_attention(c.tree, c.pages, c.q, c.k, c.v, c.kp, c.vp, o, c.scale, ws=ws)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_a_small_workspace_is_not_used():
    c = Case([np.array([-1], np.int32)], [3000], 2, 1, 64, 64, BF, seed=15)
    o = torch.empty_like(c.q.contiguous())
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    tgdn.paged_tree_attention(c.tree, c.pages, c.q, c.k, c.v, c.kp, c.vp, o, c.scale, ws=ws)
    c.check(o)
    assert not bool(ws.any())
