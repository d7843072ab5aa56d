"""Prompt and paged attention with large logits and row maxima that move from tile to tile, held to
the tolerance of ordinary ones.

q and k are whole numbers times powers of two, so every score is exact in fp32 and only the
exponent is rounded: of c x - c m (c = scale log2(e)) the kernels round c, c m and the result, each
by 2^-24 of itself, and a rescaling does so once more: a probability is off by at most
    4 ln(2) 2^-24 max|c x|  <=  4 ln(2) 2^-24 (512 log2(e))  =  1.3e-4  <  2^-12
of itself, which is the share that attend()'s tolerance has for fp32 work.  No slack is added, and
zeros, or one key's value in place of another's, would not pass (checked)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from attn_helpers import assert_within, attend, visible_tree  # noqa: E402
from test_gpu_paged_tree_attention import BF, HF, Case, trees  # noqa: E402
from test_gpu_prompt_attention import make, run  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402

SHAPES = ["drawn", "rising", "falling", "last tile", "flat"]


def whole(x, g, top):
    x.copy_(torch.randint(-top, top + 1, x.shape, generator=g))


def shape_keys(k, kind):
    """k [positions][H_kv][d] of whole numbers, scaled by powers of two position by position."""
    n = k.shape[0]
    at = torch.arange(n)
    up = {"drawn": torch.zeros(n), "rising": (at * 6 // max(n, 1)).float() - 5,
          "falling": -(at * 6 // max(n, 1)).float(), "last tile": torch.where(at >= n - 100, 0.0, -4.0),
          "flat": torch.full((n,), -12.0)}[kind]
    k.mul_(torch.exp2(up).to(k.dtype).to(k.device)[:, None, None])


def held(got, ref, tol, q, kind):
    assert_within(got, ref, tol)
    if kind != "flat":  # (flat ones average hundreds of values to nearly nothing)
        assert float((tol < 0.1 * ref.abs()).double().mean()) > 0.8
    assert bool(((torch.roll(ref, 1, -1) - ref).abs() > tol).double().mean() > 0.8)


@pytest.mark.parametrize("kind", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,H_q,H_kv,d", [([400], 2, 1, 64), ([700], 4, 1, 128), ([1300], 2, 2, 64),
                                             ([900], 1, 1, 128), ([300, 80], 3, 1, 96)])
def test_prompts(lens, H_q, H_kv, d, dtype, kind):
    cu, q, k, v = make(lens, H_q, H_kv, d, dtype, seed=d)
    g = torch.Generator().manual_seed(3)
    whole(q, g, 4), whole(k, g, 4)
    scale = 1.0 if d == 64 else 0.5
    at = 0
    for n in lens:
        shape_keys(k[at:at + n], kind)
        at += n
    largest = scale * float(torch.einsum("qhd,khd->hqk", q[:, :H_kv].double(), k.double()).abs().max())
    assert largest <= 512 and (kind == "flat" or largest > 60)
    o, st = run(cu, q, k, v, scale)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        ref, tol = attend(q[s], k[s], v[s], np.tril(np.ones((n, n), bool)), scale)
        held(o[s], ref, tol, q, kind)
        at += n


@pytest.mark.parametrize("kind", SHAPES)
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("nodes,lens,H_q,H_kv,d,dtype", [
    ([33, 7], [2100, 900], 4, 1, 128, BF), ([1, 2], [5000, 130], 4, 2, 64, HF), ([64], [1500], 4, 1, 96, HF)])
def test_trees(nodes, lens, H_q, H_kv, d, dtype, split, kind):
    c = Case(trees(np.random.default_rng(4), nodes), lens, H_q, H_kv, d, 32, dtype, seed=5)
    g = torch.Generator().manual_seed(6)
    whole(c.q, g, 4), whole(c.k, g, 4)
    c.scale = 1.0 if d == 64 else 0.5
    for b, n in enumerate(lens):
        rows = torch.randint(-4, 5, (n, H_kv, d), generator=g).to(dtype).cuda()
        shape_keys(rows, kind)
        page = c.pages.table[b].long()
        for i in range(0, n, c.ps):
            c.kp[page[i // c.ps], :, :min(c.ps, n - i)] = rows[i:i + c.ps].transpose(0, 1)
    if kind == "flat":
        c.k.mul_(2.0 ** -12)
    o = c.run(split)
    for b, p in enumerate(c.parents):
        s = slice(int(c.cu[b]), int(c.cu[b + 1]))
        k, v = c.keys(b)
        see = np.concatenate([np.ones((len(p), lens[b]), bool), visible_tree(p)], 1)
        ref, tol = attend(c.q[s], k, v, see, c.scale)
        held(o[s], ref, tol, c.q[s], kind)


def test_the_statement_refuses_zeros():
    cu, q, k, v = make([400], 2, 1, 64, HF, seed=64)
    g = torch.Generator().manual_seed(3)
    whole(q, g, 4), whole(k, g, 4)
    ref, tol = attend(q, k, v, np.tril(np.ones((400, 400), bool)), 1.0)
    with pytest.raises(AssertionError):
        assert_within(torch.zeros_like(ref), ref, tol)
