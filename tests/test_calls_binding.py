"""The C++ part of the binding (csrc/binding.cpp) refuses, without a GPU, what must not reach a
kernel, and never lets a C++ exception or a bad argument count end the process."""
import pytest

torch = pytest.importorskip("torch")
from tree_speculative_decoding_gated_gb300 import build, tgdn  # noqa: E402

CALLS = {"rope": 12, "prompt_attention": 9, "pages_reserve": 4, "pages_append": 9, "pages_fork": 7,
         "pages_free": 3, "pages_compact": 5, "paged_tree_attention": 11}


@pytest.fixture(scope="module")
def native():
    build.build()
    return tgdn._native()


@pytest.mark.parametrize("name", CALLS)
def test_argument_counts(native, name):
    for n in (0, CALLS[name] - 1, CALLS[name] + 1):
        with pytest.raises(TypeError, match="arguments"):
            getattr(native, name)(*[None] * n)
    with pytest.raises((TypeError, AttributeError)):
        getattr(native, name)(*[None] * CALLS[name])


def test_host_tensors_are_refused(native):
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    freq, _ = tgdn.rope_freqs(64, device="cpu")
    with pytest.raises(ValueError, match="q: must be a CUDA tensor"):
        tgdn.rope(q, None, q, None, freq, cu=cu)
    with pytest.raises(ValueError, match="q: must be a CUDA tensor"):
        tgdn.prompt_attention(cu, q, q, q, q, 0.1, cu)
    pages = tgdn.Pages(2, 4, 16, 2, device="cpu")
    with pytest.raises(ValueError, match="table: must be a CUDA tensor"):
        tgdn.pages_free(pages, cu)


def test_types_and_dimensions(native):
    cu = torch.tensor([0, 3], dtype=torch.int32)
    for q in (3, None, torch.zeros((3, 64)), torch.zeros((3, 2, 64), dtype=torch.float64)):
        with pytest.raises(TypeError, match="q: expected a float32, bfloat16 or float16 tensor"):
            tgdn.rope(q, None, q, None, cu, cu=cu)
    q = torch.zeros((3, 2, 64))
    with pytest.raises(TypeError, match="cu: expected a torch.Tensor"):
        tgdn.rope(q, None, q, None, cu, cu=[0, 3])
    with pytest.raises(ValueError, match="k: shape"):
        tgdn.rope(q, torch.zeros(3), q, None, cu, cu=cu)


def test_objects_without_the_fields(native):
    class Some:
        B = "two"
    with pytest.raises(AttributeError, match="B"):
        tgdn.pages_free(object(), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        tgdn.pages_free(Some(), torch.zeros(1, dtype=torch.int32))
