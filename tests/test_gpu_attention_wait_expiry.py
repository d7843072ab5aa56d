"""A bounded device wait of the attention kernels that runs out: the queries of one sequence's
head never come (tgdn_debug_set_wait_hooks), so the CTAs that hold its items stop with others
known ahead and still to come: when the copies have no room any more (a limit of a few ms), or,
where there is nothing left to copy, when the products' wait runs out (2 s).  No fault and no hang: the call returns, every
sequence whose status is TGDN_SEQ_OK matches the 64-bit statement, the withheld one is
TGDN_SEQ_TIMEOUT, and the next call is right."""
import time

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from attn_helpers import assert_within, attend  # noqa: E402
from test_gpu_paged_tree_attention import BF, HF, Case, trees  # noqa: E402
from test_gpu_prompt_attention import check, make, run  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402

LIMIT_NS = 5_000_000
MOST = 3.0  # seconds: the longer limit and the work


def withheld(item, call):
    """The call with the item's queries withheld, and what it took."""
    call()  # (the kernel is loaded)
    try:
        tgdn.debug_set_wait_hooks(LIMIT_NS, item)
        began = time.time()
        out = call()
        return out, time.time() - began
    finally:
        tgdn.debug_set_wait_hooks()


# many short prompts (several items of different sequences per CTA, known ahead), uneven ones of
# two row tiles, long ones whose key tiles go to both pipelines in turn
@pytest.mark.parametrize("lens,H_q,H_kv,d,dtype", [
    ([1 + 7 * i % 40 for i in range(500)], 4, 4, 64, BF),
    ([1 + 7 * i % 40 for i in range(500)], 8, 4, 128, HF),
    ([300 + 37 * i % 200 for i in range(60)], 16, 4, 128, BF),
    ([1100, 900, 800], 8, 2, 64, HF), ([1100, 900, 800], 4, 2, 128, BF),
    ([700] * 30, 12, 4, 96, BF)])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_prompts(lens, H_q, H_kv, d, dtype, where):
    cu, q, k, v = make(lens, H_q, H_kv, d, dtype, seed=1)
    b = int(where * (len(lens) - 1))
    (o, st), took = withheld(b * H_kv + H_kv - 1, lambda: run(cu, q, k, v, d ** -0.5))
    st = st.tolist()
    assert took < MOST and set(st) <= {tgdn.SEQ_OK, tgdn.SEQ_TIMEOUT} and st[b] == tgdn.SEQ_TIMEOUT
    at = np.r_[0, np.cumsum(lens)]
    for i, n in enumerate(lens):
        if st[i] == tgdn.SEQ_OK:
            s = slice(int(at[i]), int(at[i + 1]))
            ref, tol = attend(q[s], k[s], v[s], np.tril(np.ones((n, n), bool)), d ** -0.5)
            assert_within(o[s], ref, tol, f"sequence {i}")
    assert st.count(tgdn.SEQ_OK) >= (len(lens) - 20 if max(lens) <= 64 else 0)  # (an item each)
    o, st = run(cu, q, k, v, d ** -0.5)
    assert not any(st.tolist())
    check(lens, q, k, v, d ** -0.5, o)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("nodes,lens,H_q,H_kv,d,ps", [
    ([3] * 200, [40 + 13 * i % 90 for i in range(200)], 4, 4, 64, 16),      # many items per CTA
    ([9] * 50, [900 + 31 * i % 400 for i in range(50)], 8, 4, 128, 64),    # cut items among whole
    ([33, 12, 0, 5], [9000, 6001, 50, 0], 4, 1, 128, 64),                  # items of many parts
    ([129] * 12, [700] * 12, 8, 2, 96, 32)])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_trees(nodes, lens, H_q, H_kv, d, ps, where, split):
    B = len(nodes)
    c = Case(trees(np.random.default_rng(2), nodes), lens, H_q, H_kv, d, ps, BF, seed=3)
    b = int(where * (B - 1))

    def call():
        tgdn.tree_prep(c.tree)
        return c.run(split)

    o, took = withheld(b * H_kv, call)
    st = c.tree.status.tolist()
    assert took < MOST and set(st) <= {tgdn.SEQ_OK, tgdn.SEQ_TIMEOUT}
    assert st[b] == tgdn.SEQ_TIMEOUT
    c.check(o, skip=[i for i in range(B) if st[i] != tgdn.SEQ_OK])
    assert st.count(tgdn.SEQ_OK) >= (B - 20 if B > 40 else 0)
    tgdn.tree_prep(c.tree)
    c.check(c.run(split))
    assert not any(c.tree.status.tolist())


def test_the_limit_alone_changes_nothing():
    lens = [700, 1, 513, 900]
    cu, q, k, v = make(lens, 8, 2, 128, BF, seed=5)
    want, _ = run(cu, q, k, v, 0.088)
    (o, st), _ = withheld(-1, lambda: run(cu, q, k, v, 0.088))
    assert not any(st.tolist()) and torch.equal(o, want)
