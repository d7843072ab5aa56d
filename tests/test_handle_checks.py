"""The C struct behind a tree or a cache is checked anew when a tensor was changed in place, also
at the same address: made smaller, transposed, given other strides, another type."""
import pytest

torch = pytest.importorskip("torch")
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402


def counted(cls, *args, **kw):
    made = []

    class Counted(cls):
        def _make(self):
            made.append(1)
            return object()

    return Counted(*args, **kw), made


@pytest.mark.parametrize("change", [
    lambda p: p.len.resize_(1), lambda p: p.table.t_(), lambda p: p.refs.as_strided_((2,), (2,)),
    lambda p: p.table.resize_(2, 1), lambda p: setattr(p.held, "data", p.held.view(torch.float32))])
def test_changes_at_the_same_address(change):
    pages, made = counted(tgdn.Pages, 2, 4, 16, 3, device="cpu")
    a = pages.c()
    assert pages.c() is a and len(made) == 1
    before = [getattr(pages, n).data_ptr() for n in pages._tensors]
    change(pages)
    assert [getattr(pages, n).data_ptr() for n in pages._tensors] == before
    assert pages.c() is not a and len(made) == 2
    assert len({id(pages.c()) for _ in range(3)}) == 1 and len(made) == 2


def test_a_tree_likewise():
    cu, parent = (torch.tensor(x, dtype=torch.int32) for x in ([0, 2], [-1, 0]))
    tree, made = counted(tgdn.Tree, cu, parent, 2, 4)
    tree.c()
    tree.c()
    assert len(made) == 1
    tree.parent.resize_(1)
    tree.c()
    assert len(made) == 2


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_a_shrunken_tensor_is_refused():
    tree = tgdn.Tree.from_host([0, 3], [-1, 0, 0], 3, 4)
    tgdn.tree_prep(tree)
    tree.parent.resize_(2)
    with pytest.raises(ValueError, match="parent"):
        tgdn.tree_prep(tree)
    tree.parent.resize_(3)
    tree.status.as_strided_((1,), (1,))
    tgdn.tree_prep(tree)
    pages = tgdn.Pages(2, 4, 16, 3)
    pages.c()
    pages.table.t_()
    with pytest.raises(ValueError, match="table"):
        tgdn.pages_workspace_bytes(pages)
