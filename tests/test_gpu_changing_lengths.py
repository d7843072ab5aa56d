"""Cached lengths that another stream changes while tgdn_paged_tree_attention reads them.  The
page calls of one cache belong on one stream, so such a call's outputs are anything; but it
ends, touches nothing outside its arrays, and the next call is right."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from test_gpu_paged_tree_attention import BF, Case, ints, trees  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402


def race(before, after, rounds=80):
    """Calls that begin with the lengths `before`, which become `after` at about the same time.
    More than 32 sequences: those past the first 32 are read a second time."""
    rng = np.random.default_rng(0)
    B = 100
    full = rng.integers(300, 900, B)
    c = Case(trees(rng, rng.integers(1, 6, B)), full.tolist(), 4, 2, 64, 16, BF, seed=1)
    ends = [ints(full * x) for x in (before, after)]
    nb = tgdn.paged_tree_attention_workspace_bytes(c.tree, c.pages, 4, 2, 64)
    ws, o = torch.zeros(nb, dtype=torch.uint8, device="cuda"), torch.empty_like(c.q.contiguous())
    main, side, gate = (torch.cuda.Stream() for _ in range(3))
    for i in range(rounds):
        c.pages.len.copy_(ends[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(gate):
            torch.cuda._sleep(200_000)
            both = gate.record_event()
        main.wait_event(both)
        side.wait_event(both)
        with torch.cuda.stream(main):
            tgdn.paged_tree_attention(c.tree, c.pages, c.q, c.k, c.v, c.kp, c.vp, o, c.scale,
                                      ws=ws if i % 4 else None)
        with torch.cuda.stream(side):
            for _ in range(i % 7):
                c.pages.status.zero_()  # (a little later each time)
            c.pages.len.copy_(ends[1])
        torch.cuda.synchronize()
    assert c.tree.status.tolist() == [0] * B
    c.pages.len.copy_(ints(full))
    c.check(c.run())


def test_lengths_that_shrink_under_way():
    race(1, 0)


def test_lengths_that_grow_under_way():
    race(0, 1)
