"""The attention-layer calls together (examples/attention_decode.py): prefill, forks, draft
trees over the paged cache, accepted paths appended, freeing and compaction.

Every generated token is held against the decoder in 64 bits on the same tokens: its logit
may lie below the largest by the roundings at most.  A token passes 16 roundings to bf16 in
two layers (norm, projection, rotation, probabilities, attention output, its projection and
the residual sum of each; the last norm and the logits), each of at most 2^-8 of a value
whose share of a logit stays below 4.5 here, for each of two logits: 2 * 16 * 2^-8 * 4.5.
A token drawn at random lies about 3 below."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from attn_helpers import inv_freq, rotate  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MARGIN = 2 * 16 * 2.0 ** -8 * 4.5


def example():
    spec = importlib.util.spec_from_file_location(
        "attention_decode", os.path.join(ROOT, "examples", "attention_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def logits64(model, tokens):
    """Every position's logits, in 64 bits from the stored weights."""
    w = lambda t: t.detach().cpu().double()  # noqa: E731
    norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    n = len(tokens)
    x = w(model.embed)[torch.tensor(tokens)]
    f, _ = inv_freq(model.d, 10000.0)
    see = np.tril(np.ones((n, n), bool))
    H_q, H_kv, d = model.H_q, model.H_kv, model.d
    for w_qkv, w_o in zip(model.w_qkv, model.w_o):
        q, k, v = (norm(x) @ w(w_qkv)).view(n, -1, d).split([H_q, H_kv, H_kv], dim=1)
        q, k = (rotate(t, np.arange(n), f, 1.0, False)[0] for t in (q, k))
        o = torch.empty_like(q)
        for h in range(H_q):
            s = d ** -0.5 * q[:, h] @ k[:, h // (H_q // H_kv)].T
            s = s.masked_fill(~torch.as_tensor(see), -float("inf"))
            o[:, h] = torch.softmax(s, -1) @ v[:, h // (H_q // H_kv)]
        x = x + o.reshape(n, -1) @ w(w_o)
    return norm(x) @ w(model.head)


@pytest.mark.parametrize("sizes", [
    dict(H_q=8, H_kv=2, d=64, page_size=16),
    dict(H_q=6, H_kv=1, d=128, page_size=64, n_pages=64, max_pages=8)])
def test_prefill_trees_and_cache(sizes):
    answers, count, lengths = 2, 24, (150, 37, 1, 130)
    out = example().run(lengths=lengths, answers=answers, count=count, **sizes)
    for r in out.values():
        model = r["model"]
        for b, tokens in enumerate(r["tokens"]):
            prompt = r["prompts"][b % len(lengths)]
            got = logits64(model, prompt + tokens[:-1])[len(prompt) - 1:]
            below = got.max(-1).values - got.gather(-1, torch.tensor(tokens)[:, None])[:, 0]
            assert float(below.max()) <= MARGIN, (b, below)
        # the first answer's pages are what is left, in front
        held = -(-(lengths[0] + len(r["tokens"][0]) - 1) // model.pages.page_size)
        assert held <= r["live_pages"] <= held + 1
        assert model.pages.len.tolist() == [lengths[0] + len(r["tokens"][0]) - 1] + \
            [0] * (model.pages.B - 1)
        assert int((model.pages.refs > 0).sum()) == r["live_pages"]
        assert bool((model.pages.refs[r["live_pages"]:] == 0).all())
    assert out["token by token"]["steps"] == count - 1
    assert out["draft trees"]["steps"] < out["token by token"]["steps"]
