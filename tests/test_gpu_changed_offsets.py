"""Tree offsets that are overwritten after tgdn_tree_prep: tgdn_paged_tree_attention looks at them
again, and rows of a range that is not one are neither read nor written."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import numpy as np  # noqa: E402

from test_gpu_paged_tree_attention import BF, Case, ints, trees  # noqa: E402

MAX, MIN = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("cu", [[0, 5, MAX, MIN, 14], [0, 5, MAX, MIN + 2, MAX], [0, 5, MIN, MAX, MIN + 3],
                                [0, 5, 1 << 30, -1 << 30, -(1 << 30) + 1]])
@pytest.mark.parametrize("split", [False, True])
def test_offsets_at_the_ends_of_int32(cu, split):
    c = Case(trees(np.random.default_rng(1), [5, 3, 4, 2]), [700, 40, 900, 30], 4, 2, 64, 16, BF, seed=1)
    good = c.run(split)
    c.tree.cu_nodes.copy_(ints(cu))
    o = c.run(split)
    assert torch.allclose(o[:5].float(), good[:5].float(), atol=2.0 ** -6)
    assert bool(torch.isnan(o[5:]).all())
    assert c.tree.status.tolist()[0] == 0
