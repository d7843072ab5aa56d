"""The attention layers' calls refuse tensors of a device that is not the current one: the launch
goes to the current device, whose kernels would follow foreign pointers.  Tensors without storage
stand for those of a second device, so nothing here needs a GPU, let alone two."""
import pytest

torch = pytest.importorskip("torch")
from tree_speculative_decoding_gated_gb300 import build, tgdn  # noqa: E402

I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def native():
    build.build()
    return tgdn._native()


class Bare(torch.Tensor):
    """A tensor of a device without storage."""

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


def at(shape, dtype, device="cuda:1"):
    shape = (shape,) if isinstance(shape, int) else shape
    return torch.Tensor._make_wrapper_subclass(Bare, shape, dtype=dtype, device=device)


def test_another_device():
    q, k, cu, word = at((3, 4, 64), BF), at((3, 2, 64), BF), at((2,), I32), at((4096,), torch.uint8)
    with pytest.raises(ValueError, match="q: on cuda:1, the current device is cuda:0"):
        tgdn.rope(q, None, q, None, at((32,), torch.int64), cu=cu)
    with pytest.raises(ValueError, match="q: on cuda:1"):
        tgdn.prompt_attention(cu, q, k, k, q, 0.1, cu)
    pages = tgdn.Pages(1, 4, 16, 2, device="cpu")
    for n, shape in dict(table=(1, 2), len=1, held=1, refs=4, status=1).items():
        setattr(pages, n, at(shape, I32))
    pool, one = at((1, 2, 4, 2, 16, 64), BF), at((1,), I32)
    for call in (lambda: tgdn.pages_reserve(pages, one, word), lambda: tgdn.pages_free(pages, one),
                 lambda: tgdn.pages_append(pages, cu, k, k, pool),
                 lambda: tgdn.pages_fork(pages, one, one, pool, one, word),
                 lambda: tgdn.pages_compact(pages, pool, one, word)):
        with pytest.raises(ValueError, match="table: on cuda:1"):
            call()


def test_one_tensor_of_another_device():
    here = lambda *a: at(*a, device="cuda:0")  # noqa: E731
    q, k, cu = here((3, 4, 64), BF), here((3, 2, 64), BF), here((2,), I32)
    for name, args in dict(cu=(at((2,), I32), q, k, k, q), k=(cu, q, at((3, 2, 64), BF), k, q),
                           v=(cu, q, k, at((3, 2, 64), BF), q),
                           o=(cu, q, k, k, at((3, 4, 64), BF))).items():
        with pytest.raises(ValueError, match=f"^{name}: on cuda:1"):
            tgdn.prompt_attention(*args, 0.1, here((1,), I32))
    with pytest.raises(ValueError, match="^status: on cuda:1"):
        tgdn.prompt_attention(cu, q, k, k, q, 0.1, at((1,), I32))
