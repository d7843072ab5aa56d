"""The paged cache against a plain model that keeps every sequence's rows in a list: random
runs of reserve, append (prompts, accepted paths, layer by layer), fork, free and compact, with
the bookkeeping equal number for number and every sequence's rows equal bit for bit; the order
in which pages are given out; refusals that only the device sees; sizes at the edges."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402

OK, BAD_RANGE, BAD_PAGE, NO_PAGES = 0, 7, 8, 9


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Model:
    """Pages as lists; rows as (key, value) integers per position."""

    def __init__(self, B, n_pages, ps, max_pages):
        self.B, self.n, self.ps, self.cols = B, n_pages, ps, max_pages
        self.pages = [[] for _ in range(B)]
        self.rows = [[] for _ in range(B)]
        self.refs = [0] * n_pages

    def free_pages(self):
        return [p for p in range(self.n) if self.refs[p] == 0]

    def reserve(self, add):
        free, asked, st = self.free_pages(), 0, []
        for b in range(self.B):
            need = -(-(len(self.rows[b]) + add[b]) // self.ps)
            lack = max(0, need - len(self.pages[b]))
            if add[b] < 0:
                st.append(BAD_PAGE)
            elif need > self.cols:
                st.append(NO_PAGES)
            elif lack and asked + lack > len(free):
                asked += lack
                st.append(NO_PAGES)
            else:
                for p in free[asked:asked + lack]:
                    self.pages[b].append(p)
                    self.refs[p] = 1
                asked += lack
                st.append(OK)
        return st

    def append(self, b, rows):
        if len(self.rows[b]) + len(rows) > len(self.pages[b]) * self.ps:
            return NO_PAGES
        self.rows[b] += rows
        return OK

    def fork(self, src, dst):
        before = [list(r) for r in self.rows]
        held = [list(p) for p in self.pages]
        free, asked, st, seen = self.free_pages(), 0, [], set()
        for x, y in zip(src, dst):
            ok = 0 <= x < self.B and 0 <= y < self.B and not held[y] and y not in seen
            seen.add(y)
            if not ok:
                st.append(BAD_PAGE)
                continue
            full, tail = divmod(len(before[x]), self.ps)
            if tail and asked >= len(free):
                asked += 1
                st.append(NO_PAGES)
                continue
            self.pages[y] = held[x][:full]
            for p in self.pages[y]:
                self.refs[p] += 1
            if tail:
                self.pages[y].append(free[asked])
                self.refs[free[asked]] = 1
                asked += 1
            self.rows[y] = list(before[x])
            st.append(OK)
        return st

    def release(self, seqs):
        for b in seqs:
            if 0 <= b < self.B:
                for p in self.pages[b]:
                    self.refs[p] -= 1
                self.pages[b], self.rows[b] = [], []

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        movers = [p for p in range(live, self.n) if self.refs[p]]
        holes = [p for p in range(live) if not self.refs[p]]
        to = dict(zip(movers, holes))
        for b in range(self.B):
            self.pages[b] = [to.get(p, p) for p in self.pages[b]]
        for p, h in to.items():
            self.refs[h], self.refs[p] = self.refs[p], 0
        return live


class Cache:
    def __init__(self, B, n_pages, ps, max_pages, L, H_kv, d, dtype):
        self.m = Model(B, n_pages, ps, max_pages)
        self.p = tgdn.Pages(B, n_pages, ps, max_pages)
        self.pool = self.p.pool(L, H_kv, d, dtype)
        self.pool.fill_(float("nan"))
        self.ws = torch.full_like(tgdn.pages_workspace(self.p), 255)   # stale bytes
        self.L, self.H, self.d, self.dtype = L, H_kv, d, dtype
        self.made = 0

    def new_rows(self, T):
        """T rows whose every element tells its row: k, v [L][T][H][d]."""
        ids = torch.arange(self.made, self.made + T)
        self.made += T
        e = torch.arange(self.d)[None, None, None] * 3 + torch.arange(self.H)[None, None, :, None] * 7
        base = (ids[None, :, None, None] * 5 + torch.arange(self.L)[:, None, None, None] * 11 + e) % 250
        k = base.to(self.dtype).cuda()
        v = (-base - 1).to(self.dtype).cuda()
        return ids.tolist(), k, v

    def expect(self, ids):
        e = torch.arange(self.d)[None, None, None] * 3 + torch.arange(self.H)[None, None, :, None] * 7
        base = (torch.tensor(ids, dtype=torch.long)[None, :, None, None] * 5 +
                torch.arange(self.L)[:, None, None, None] * 11 + e) % 250
        return base.to(self.dtype), (-base - 1).to(self.dtype)

    def check(self):
        torch.cuda.synchronize()
        m, p = self.m, self.p
        assert p.len.tolist() == [len(r) for r in m.rows]
        assert p.held.tolist() == [len(x) for x in m.pages]
        assert p.refs.tolist() == m.refs
        table = p.table.tolist()
        pool = self.pool.cpu()
        for b in range(m.B):
            assert table[b][:len(m.pages[b])] == m.pages[b], b
            if m.rows[b]:
                ids = torch.tensor(m.pages[b])
                got = pool[:, :, ids].permute(0, 1, 2, 4, 3, 5).reshape(
                    self.L, 2, -1, self.H, self.d)[:, :, :len(m.rows[b])]
                k, v = self.expect(m.rows[b])
                assert torch.equal(got[:, 0], k) and torch.equal(got[:, 1], v), b


def append_prompt(c, counts, advance=True):
    ids, k, v = c.new_rows(max(sum(counts), 1))
    cu = np.r_[0, np.cumsum(counts)]
    tgdn.pages_append(c.p, ints(cu), k, v, c.pool, advance=advance)
    st = [c.m.append(b, ids[cu[b]:cu[b + 1]]) for b in range(c.m.B)] if advance else None
    return st


def append_path(c, rng, counts):
    rows = [int(n + rng.integers(0, 5)) for n in counts]
    ids, k, v = c.new_rows(max(sum(rows), 1))
    cu = np.r_[0, np.cumsum(rows)]
    path = np.full((c.m.B, 12), -1, np.int32)
    for b, n in enumerate(counts):
        path[b, :n] = np.sort(rng.choice(rows[b], n, replace=False)) if n else []
    tgdn.pages_append(c.p, ints(cu), k, v, c.pool, path=ints(path), n_path=ints(counts))
    return [c.m.append(b, [ids[cu[b] + i] for i in path[b, :n]]) for b, n in enumerate(counts)]


@pytest.mark.parametrize("B,n_pages,ps,cols,L,H,d,dtype,seed", [
    (8, 40, 16, 9, 2, 2, 64, torch.bfloat16, 0), (5, 200, 32, 12, 1, 4, 128, torch.float16, 1),
    (40, 90, 16, 6, 3, 1, 8, torch.bfloat16, 2), (3, 12, 256, 4, 1, 3, 40, torch.float16, 3),
    (1, 5, 128, 5, 9, 1, 256, torch.bfloat16, 4)])
def test_random_runs(B, n_pages, ps, cols, L, H, d, dtype, seed):
    rng = np.random.default_rng(seed)
    c = Cache(B, n_pages, ps, cols, L, H, d, dtype)
    for step in range(30):
        what = rng.choice(["reserve", "path", "prompt", "fork", "free", "compact"],
                          p=[.2, .25, .2, .15, .12, .08])
        if what in ("reserve", "prompt", "path"):
            top = 13 if what == "path" else 3 * ps
            add = [int(x) if rng.random() < 0.5 else 0 for x in rng.integers(0, top, B)]
            if what == "reserve" and rng.random() < 0.2:
                add[int(rng.integers(B))] = -1
            tgdn.pages_reserve(c.p, ints(add), c.ws)
            assert c.p.status.tolist() == (want := c.m.reserve(add)), step
            if what != "reserve":   # sequences without room are refused by the append
                st = append_prompt(c, add) if what == "prompt" else append_path(c, rng, add)
                assert c.p.status.tolist() == st, step
        elif what == "fork":
            n = int(rng.integers(1, B + 1))
            src, dst = rng.integers(-1, B + 1, n).tolist(), rng.integers(-1, B + 1, n).tolist()
            out = torch.full((n,), -1, dtype=torch.int32, device="cuda")
            tgdn.pages_fork(c.p, ints(src), ints(dst), c.pool, out, c.ws)
            assert out.tolist() == c.m.fork(src, dst), step
        elif what == "free":
            seqs = rng.integers(-1, B + 1, int(rng.integers(1, B + 1))).tolist()   # some twice
            tgdn.pages_free(c.p, ints(seqs))
            c.m.release(seqs)
        else:
            n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
            tgdn.pages_compact(c.p, c.pool, n_live, c.ws)
            assert int(n_live) == c.m.compact(), step
            assert c.p.status.tolist() == [OK] * B
        c.check()


def test_pages_come_lowest_first_in_order_of_sequences():
    c = Cache(3, 10, 16, 4, 1, 1, 64, torch.bfloat16)
    tgdn.pages_reserve(c.p, ints([17, 0, 33]), c.ws)
    assert c.p.table[0, :2].tolist() == [0, 1] and c.p.table[2, :3].tolist() == [2, 3, 4]
    tgdn.pages_free(c.p, ints([0]))
    tgdn.pages_reserve(c.p, ints([0, 40, 0]), c.ws)
    assert c.p.table[1, :3].tolist() == [0, 1, 5]


def test_a_later_sequence_is_not_served_past_one_that_did_not_fit():
    c = Cache(4, 5, 16, 8, 1, 1, 64, torch.bfloat16)
    tgdn.pages_reserve(c.p, ints([16, 100, 16, 0]), c.ws)
    assert c.p.status.tolist() == [OK, NO_PAGES, NO_PAGES, OK] and c.p.held.tolist() == [1, 0, 0, 0]


@pytest.mark.parametrize("n_pages", [1, 31, 8191, 8192, 8193, 30000])
def test_large_pools_are_scanned_in_full(n_pages):
    """Free pages only at the end of the pool, past whole rounds of the scan."""
    p = tgdn.Pages(2, n_pages, 16, 3)
    p.refs.fill_(1)
    last = [n_pages - 1] if n_pages < 3 else [n_pages - 3, n_pages - 1]
    p.refs[last] = 0
    tgdn.pages_reserve(p, ints([1, 16]), tgdn.pages_workspace(p))
    got = [int(p.table[b, 0]) for b in range(2) if p.held[b] > 0]
    assert got == last and int(p.refs.min()) == 1


def test_many_sequences():
    B = 2500
    p = tgdn.Pages(B, 6000, 16, 2)
    add = np.random.default_rng(0).integers(0, 33, B)
    tgdn.pages_reserve(p, ints(add), tgdn.pages_workspace(p))
    want = -(-add // 16)
    assert p.held.tolist() == want.tolist()
    used = np.concatenate([p.table[b, :want[b]].cpu().numpy() for b in range(B)])
    assert used.tolist() == list(range(want.sum()))


def test_layer_by_layer_appends():
    """advance=False for all layers but the last: as one call for all of them."""
    c = Cache(3, 20, 16, 5, 1, 2, 64, torch.bfloat16)
    tgdn.pages_reserve(c.p, ints([20, 0, 33]), c.ws)
    c.m.reserve([20, 0, 33])
    ids, k, v = c.new_rows(53)
    cu = ints([0, 20, 20, 53])
    other = torch.full_like(c.pool, float("nan"))
    tgdn.pages_append(c.p, cu, k[0], v[0], other, advance=False)
    assert c.p.len.tolist() == [0, 0, 0] and c.p.status.tolist() == [0, 0, 0]
    tgdn.pages_append(c.p, cu, k, v, c.pool)
    c.m.append(0, ids[:20]), c.m.append(2, ids[20:])
    c.check()
    assert torch.equal(other.view(torch.int16), c.pool.view(torch.int16))


def test_append_takes_views_of_a_fused_projection():
    c = Cache(1, 8, 16, 4, 1, 2, 64, torch.float16)
    tgdn.pages_reserve(c.p, ints([30]), c.ws)
    c.m.reserve([30])
    ids, k, v = c.new_rows(30)
    qkv = torch.randn(30, 9, 64, device="cuda").half()
    qkv[:, 5:7], qkv[:, 7:9] = k[0], v[0]
    tgdn.pages_append(c.p, ints([0, 30]), qkv[:, 5:7], qkv[:, 7:9], c.pool)
    c.m.append(0, ids)
    c.check()


def test_what_only_the_device_sees():
    c = Cache(4, 12, 16, 3, 1, 1, 64, torch.bfloat16)
    tgdn.pages_reserve(c.p, ints([16, 16, 16, 16]), c.ws)
    c.m.reserve([16, 16, 16, 16])
    ids, k, v = c.new_rows(10)
    path = ints([[0, 9, -1], [0, 1, 2], [0, 1, -1], [0, -1, -1]])
    # a node outside the tree, a count above the path's width, a row range past T, a good one
    tgdn.pages_append(c.p, ints([0, 3, 6, 6, 10]), k, v, c.pool, path=path, n_path=ints([2, 4, 1, 1]))
    assert c.p.status.tolist() == [BAD_RANGE, BAD_RANGE, BAD_RANGE, OK]
    c.m.append(3, [ids[6]])
    tgdn.pages_append(c.p, ints([0, 3, 2, 2, 40]), k, v, c.pool)
    assert c.p.status.tolist() == [OK, BAD_RANGE, OK, BAD_RANGE]
    c.m.append(0, ids[:3])
    c.check()
    # inconsistent bookkeeping is left as it is
    c.p.len[1] = 17
    before = c.p.table.clone()
    tgdn.pages_reserve(c.p, ints([0, 5, 0, 0]), c.ws)
    assert c.p.status.tolist() == [OK, BAD_PAGE, OK, OK] and torch.equal(before, c.p.table)
    c.p.len[1] = 0
    # page numbers outside the pool are neither read nor written
    c.p.table[1, 0] = 12
    c.p.table[2, 0] = -1
    tgdn.pages_append(c.p, ints([0, 0, 1, 2, 2]), k, v, c.pool)
    assert c.p.status.tolist() == [OK, BAD_PAGE, BAD_PAGE, OK] and c.p.len.tolist() == [3, 0, 0, 1]
    out = ints([-1, -1])
    c.p.len[1] = 5
    tgdn.pages_free(c.p, ints([0]))
    tgdn.pages_fork(c.p, ints([1, 3]), ints([0, 0]), c.pool, out, c.ws)
    assert out.tolist() == [BAD_PAGE, BAD_PAGE] and c.p.held.tolist()[0] == 0
    tgdn.pages_free(c.p, ints([1, 2]))
    assert c.p.status.tolist()[1:3] == [BAD_PAGE, BAD_PAGE] and c.p.held.tolist() == [0, 0, 0, 1]


def test_fork_shares_full_pages_and_copies_the_last():
    c = Cache(4, 16, 16, 4, 2, 2, 64, torch.bfloat16)
    tgdn.pages_reserve(c.p, ints([35, 32, 0, 0]), c.ws)
    c.m.reserve([35, 32, 0, 0])
    append_prompt(c, [35, 32, 0, 0])
    out = ints([-1, -1])
    tgdn.pages_fork(c.p, ints([0, 1]), ints([2, 3]), c.pool, out, c.ws)
    assert out.tolist() == c.m.fork([0, 1], [2, 3]) == [OK, OK]
    assert c.p.table[2, :2].tolist() == c.p.table[0, :2].tolist()
    assert c.p.table[2, 2] != c.p.table[0, 2] and c.p.table[3, :2].tolist() == c.p.table[1, :2].tolist()
    # each goes its own way
    tgdn.pages_reserve(c.p, ints([3, 2, 5, 1]), c.ws)
    c.m.reserve([3, 2, 5, 1])
    append_path(c, np.random.default_rng(1), [3, 2, 5, 1])
    c.check()


def test_in_a_graph():
    c = Cache(2, 20, 16, 6, 1, 1, 64, torch.bfloat16)
    ids, k, v = c.new_rows(7)
    cu, add = ints([0, 3, 7]), ints([3, 4])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tgdn.pages_reserve(c.p, add, c.ws)
        tgdn.pages_append(c.p, cu, k, v, c.pool)
    for _ in range(6):
        g.replay()
        c.m.reserve([3, 4])
        c.m.append(0, ids[:3]), c.m.append(1, ids[3:])
    c.check()
