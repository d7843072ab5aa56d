"""The page calls on bookkeeping that is not sound: the sequence gets TGDN_SEQ_BAD_PAGE, reads
what it read before, and no other sequence loses a page."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from test_gpu_pages import BAD_PAGE, OK, ints  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402


def cache(held, ps=16, n_pages=None, cols=None, seed=0):
    """Sequences that hold scattered pages of distinct contents, and their rows of the table."""
    n_pages = n_pages or 3 * sum(held) + 7
    p = tgdn.Pages(len(held), n_pages, ps, cols or max(held) + 2)
    ids = np.random.default_rng(seed).permutation(n_pages)
    rows, at = [], 0
    for b, n in enumerate(held):
        rows.append(ids[at:at + n].tolist())
        at += n
        p.table[b, :n] = ints(rows[b])
        p.refs[rows[b]] = 1
    p.held.copy_(ints(held))
    p.len.copy_(ints([n * ps for n in held]))
    pool = p.pool(2, 1, 8, torch.float16)
    pool.copy_(torch.arange(pool.numel() // (ps * 8)).remainder(2000)[:, None].expand(-1, ps * 8)
               .reshape(pool.shape))
    return p, pool, rows


def contents(p, pool, b, columns):
    ids = p.table[b, columns].long()
    return pool[:, :, ids].clone()


def test_compaction_follows_every_entry_of_an_unsound_sequence():
    p, pool, rows = cache([40, 70, 3, 5, 2])
    p.len[0] = 40 * 16 + 1            # longer than its pages
    p.table[1, 2] = p.n_pages         # an entry outside the pool ...
    p.refs[rows[1][2]] = 0
    p.table[1, 33] = -5               # ... and one in the same lane's next turn
    p.refs[rows[1][33]] = 0
    p.held[3] = p.max_pages + 4       # more pages than columns
    sound = {0: list(range(40)), 1: [c for c in range(70) if c not in (2, 33)], 2: [0, 1, 2],
             3: [0, 1, 2, 3, 4], 4: [0, 1]}
    before = {b: contents(p, pool, b, c) for b, c in sound.items()}
    refs, n_live = int((p.refs > 0).sum()), ints([0])
    tgdn.pages_compact(p, pool, n_live, tgdn.pages_workspace(p))
    assert p.status.tolist() == [BAD_PAGE, BAD_PAGE, OK, BAD_PAGE, OK]
    assert int(n_live) == refs and int((p.refs > 0).sum()) == refs and not bool(p.refs[refs:].any())
    for b, c in sound.items():
        assert int(p.table[b, c].max()) < refs, b
        assert torch.equal(contents(p, pool, b, c), before[b]), b
    assert p.table[1, [2, 33]].tolist() == [p.n_pages, -5]
    assert p.len[0] == 641 and p.held[3] == p.max_pages + 4


@pytest.mark.parametrize("held", [-3, 7, 1000])
def test_free_refuses_a_count_outside_the_table(held):
    """Columns past the sequence's own pages keep old numbers, which other sequences hold now."""
    p, pool, rows = cache([2, 6, 4], cols=6)
    p.table[0, 2:] = p.table[1, :4]   # old numbers
    p.held[0] = held
    before = [x.clone() for x in (p.table, p.len, p.held, p.refs)]
    tgdn.pages_free(p, ints([0]))
    assert p.status.tolist() == [BAD_PAGE, OK, OK]
    assert all(torch.equal(a, b) for a, b in zip(before, (p.table, p.len, p.held, p.refs)))
    p.held[0] = 2
    tgdn.pages_free(p, ints([0, 2]))
    assert p.status.tolist() == [OK] * 3 and p.held.tolist() == [0, 6, 0]
    assert int(p.refs.sum()) == 6 and bool((p.refs[rows[1]] == 1).all())


def test_a_sequence_listed_again_keeps_its_status():
    p, pool, rows = cache([3, 4])
    p.table[0, 1] = p.n_pages
    tgdn.pages_free(p, ints([0] * 20000 + [1, -1, 2]))
    assert p.status.tolist() == [BAD_PAGE, OK] and p.held.tolist() == [0, 0]
    assert int(p.refs.sum()) == 1 and p.refs[rows[0][1]] == 1
    tgdn.pages_free(p, ints([0, 0]))
    assert p.status.tolist() == [OK, OK]
