"""tgdn_prompt_attention writes every sequence's status word once per launch, whichever of its CTAs
start and whichever are taken over: calls one behind another on several streams, more items than
SMs, words that hold something else before each call."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from test_gpu_prompt_attention import BF, make  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402


@pytest.mark.parametrize("lens", [[1], [130] * 80, [3, 0, 700, 20] * 30])
def test_every_word_is_written(lens):
    cu, q, k, v = make(lens, 8, 4, 64, BF, seed=1)
    ranges = cu.tolist()
    if len(lens) > 1:
        ranges[2] = 0  # the second one's range ends before it begins, the third's overlaps
    want = [0, 7, 7] + [0] * (len(lens) - 3) if len(lens) > 1 else [0]
    cu = torch.tensor(ranges, dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(3)]
    words = torch.full((90, len(lens)), -3, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q) for _ in streams]
    torch.cuda.synchronize()
    for i in range(words.shape[0]):
        tgdn.prompt_attention(cu, q, k, v, outs[i % 3], 0.125, words[i], stream=streams[i % 3])
    torch.cuda.synchronize()
    for i in range(words.shape[0]):
        assert words[i].tolist() == want, i
    assert torch.equal(outs[0][:1], outs[1][:1]) and torch.equal(outs[0][:1], outs[2][:1])
