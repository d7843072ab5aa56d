"""tgdn_prompt_attention against causal attention in 64 bits: head layouts, head sizes, both
types, lengths from nothing to several key tiles, strided rows; masked non-finite values; bad
ranges; capture into a graph and a side stream."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from attn_helpers import assert_within, attend  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402

BF, HF = torch.bfloat16, torch.float16


def make(lens, H_q, H_kv, d, dtype, seed=0, fused=False, gain=2.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    x = torch.randn((T, H_q + 2 * H_kv, d), generator=g)
    x[:, :H_q] *= gain
    x = x.to(dtype).cuda()
    q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = torch.tensor(np.r_[0, np.cumsum(lens)], dtype=torch.int32, device="cuda")
    return cu, q, k, v


def run(cu, q, k, v, scale, **kw):
    o = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    st = torch.full((cu.numel() - 1,), -5, dtype=torch.int32, device="cuda")
    tgdn.prompt_attention(cu, q, k, v, o, scale, st, **kw)
    torch.cuda.synchronize()
    return o, st


def check(lens, q, k, v, scale, o):
    at, worst = 0, 0.0
    for n in lens:
        if n:
            s = slice(at, at + n)
            ref, tol = attend(q[s], k[s], v[s], np.tril(np.ones((n, n), bool)), scale)
            worst = max(worst, assert_within(o[s], ref, tol, f"rows {at}..{at + n}"))
        at += n
    return worst


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("H_q,H_kv,d", [(1, 1, 64), (4, 1, 128), (16, 4, 128), (6, 2, 96), (8, 8, 64),
                                        (5, 1, 40), (7, 1, 8), (33, 1, 72), (128, 1, 16), (12, 4, 128)])
def test_ragged_batches(H_q, H_kv, d, dtype):
    lens = [1, 0, 3, 127, 128, 129, 300, 2, 0, 65]
    cu, q, k, v = make(lens, H_q, H_kv, d, dtype, seed=H_q + d, fused=(H_q in (4, 6, 8, 12)))
    o, st = run(cu, q, k, v, d ** -0.5)
    assert st.tolist() == [0] * len(lens)
    print("worst share of the tolerance", check(lens, q, k, v, d ** -0.5, o))


@pytest.mark.parametrize("lens", [[1], [2], [64], [255], [256], [257], [511], [640], [1025]])
def test_single_prompts(lens):
    cu, q, k, v = make(lens, 4, 2, 128, BF, seed=lens[0])
    o, _ = run(cu, q, k, v, 0.088)
    check(lens, q, k, v, 0.088, o)


def test_many_items_per_cta():
    """More work items than SMs: the stream of items, both row tiles, and the ring of copies."""
    lens = [700, 1, 513, 900, 64, 1100]
    cu, q, k, v = make(lens, 16, 8, 128, BF, seed=5)
    o, _ = run(cu, q, k, v, 0.088)
    check(lens, q, k, v, 0.088, o)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("H_q,H_kv,d", [(1, 1, 128), (8, 1, 64), (4, 4, 96), (2, 1, 40)])
@pytest.mark.parametrize("lens", [[768], [1024], [1100, 900], [769, 1, 2000], [1537, 1000, 0]])
def test_few_long_prompts(lens, H_q, H_kv, d, dtype):
    """One row tile per item, key tiles in turn to both pipelines (even and odd counts, items of
    one and two key tiles next to long ones)."""
    cu, q, k, v = make(lens, H_q, H_kv, d, dtype, seed=sum(lens) + d, fused=d == 96)
    o, st = run(cu, q, k, v, d ** -0.5)
    assert st.tolist() == [0] * len(lens)
    check(lens, q, k, v, d ** -0.5, o)
    again, _ = run(cu, q, k, v, d ** -0.5)
    assert torch.equal(o, again)


@pytest.mark.parametrize("at", [0, 130, 700, 899])
def test_one_pipeline_holds_all_the_weight(at):
    """A key that outweighs every other one, in either pipeline's tiles; rows before it see none
    of it."""
    cu, q, k, v = make([900], 2, 1, 128, HF, seed=21)
    q[:] = 0.5
    k[:] = 0.25 * torch.sign(k)
    k[at] = 4.0
    o, _ = run(cu, q, k, v, 0.3)
    check([900], q, k, v, 0.3, o)


def test_non_finite_values_in_either_pipeline():
    cu, q, k, v = make([1000], 2, 1, 64, BF, seed=22)
    v[333, 0, 5] = float("nan")
    v[600, 0, 9] = float("inf")
    o, _ = run(cu, q, k, v, 0.1)
    assert bool(torch.isfinite(o[:333]).all())
    assert bool(torch.isnan(o[333:, :, 5]).all()) and bool(torch.isfinite(o[:600, :, 9]).all())
    assert bool((o[600:, :, 9] == float("inf")).all())
    keep = [c for c in range(64) if c not in (5, 9)]
    assert bool(torch.isfinite(o[:, :, keep]).all())


@pytest.mark.parametrize("gain,scale", [(30.0, 0.088), (0.0, 1.0), (2.0, 1e-4), (200.0, 0.3)])
def test_peaked_and_flat_softmax(gain, scale):
    """Large logits (the running maximum moves over many tiles) and flat ones.  The tolerance
    for fp32 work grows with the logits: scale sum |q k| d 2^-23 per probability."""
    lens = [400]
    cu, q, k, v = make(lens, 2, 1, 64, HF, seed=7, gain=gain)
    o, _ = run(cu, q, k, v, scale)
    ref, tol = attend(q, k, v, np.tril(np.ones((400, 400), bool)), scale)
    logit = scale * float((q.float().abs().amax() * k.float().abs().amax()) * 64)
    A = tol / 2.0 ** -11
    assert_within(o, ref, tol + A * logit * 64 * 2.0 ** -23)


def test_the_largest_key_last():
    """Row maxima that grow tile after tile: every step rescales."""
    n = 600
    cu, q, k, v = make([n], 1, 1, 64, BF, seed=8)
    k = (torch.linspace(-1, 1, n)[:, None, None] * torch.ones(1, 1, 64)).to(BF).cuda()
    q = torch.ones_like(q) * 2
    o, _ = run(cu, q, k, v, 0.5)
    ref, tol = attend(q, k, v, np.tril(np.ones((n, n), bool)), 0.5)
    assert_within(o, ref, tol + tol * 2.0 ** 8 * 64 * 2.0 ** -23 * 64)


@pytest.mark.parametrize("d", [64, 128])
def test_masked_values_reach_no_row(d):
    """NaN and infinities in later keys and values, and in other prompts: rows before them keep
    every bit; rows that see one are not finite."""
    lens = [200, 150, 90]
    cu, q, k, v = make(lens, 4, 2, d, BF, seed=11)
    clean, _ = run(cu, q, k, v, 0.1)
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    v2[170, 0, 3] = float("nan")
    v2[199, 1, 5] = float("inf")
    k2[180, 1] = float("nan")
    k2[350 + 60] = float("inf")
    v2[350:] = float("-inf")
    q2[350 + 80] = float("nan")
    got, st = run(cu, q2, k2, v2, 0.1)
    assert st.tolist() == [0, 0, 0]
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(got[:170]), bits(clean[:170]))          # rows 0..169 of the first
    assert torch.equal(bits(got[200:350]), bits(clean[200:350]))    # the second prompt
    # heads 0, 1 read key/value head 0: only column 3 of rows 170.. is touched
    assert bool(torch.isnan(got[170:200, :2, 3]).all())
    rest = [c for c in range(d) if c != 3]
    assert torch.equal(bits(got[170:200, :2][:, :, rest].contiguous()),
                       bits(clean[170:200, :2][:, :, rest].contiguous()))
    # heads 2, 3: rows 180.. see a NaN key; row 199 the infinite value as well
    assert torch.equal(bits(got[170:180, 2:]), bits(clean[170:180, 2:]))
    assert bool(torch.isnan(got[180:200, 2:]).all())
    assert not bool(torch.isfinite(got[350:]).any())


def test_infinite_value_of_the_diagonal_tile():
    cu, q, k, v = make([100], 2, 1, 64, HF, seed=12)
    v[40, 0, 7] = float("inf")
    o, _ = run(cu, q, k, v, 0.1)
    assert bool(torch.isfinite(o[:40]).all()) and bool((o[40:, :, 7] == float("inf")).all())
    keep = [c for c in range(64) if c != 7]
    assert bool(torch.isfinite(o[40:][:, :, keep]).all())


def test_bad_ranges_are_skipped():
    cu, q, k, v = make([50, 60, 70], 2, 1, 64, BF, seed=13)
    cu2 = torch.tensor([0, 50, 40, 300], dtype=torch.int32, device="cuda")
    o, st = run(cu2, q, k, v, 0.1)
    assert st.tolist() == [0, 7, 7]
    ref, tol = attend(q[:50], k[:50], v[:50], np.tril(np.ones((50, 50), bool)), 0.1)
    assert_within(o[:50], ref, tol)
    assert bool(torch.isnan(o[50:]).all())


def test_overlapping_ranges_are_skipped():
    """More rows claimed than there are: the later claims are refused, nothing else is lost."""
    T = 700
    cu, q, k, v = make([T], 2, 1, 64, BF, seed=14)
    ranges = [0, 300, 100, 450, 0, T] + [0, T] * 40 + [T]
    cu2 = torch.tensor(ranges, dtype=torch.int32, device="cuda")
    o, st = run(cu2, q, k, v, 0.1)
    want, high = [], 0
    for lo, hi in zip(ranges[:-1], ranges[1:]):
        sound = lo <= hi
        want.append(0 if sound and lo >= high else 7)
        high = max(high, hi) if sound else high
    assert st.tolist() == want and want[0] == 0 and want[2] == 7 and want[-1] == 0
    ref, tol = attend(q[:300], k[:300], v[:300], np.tril(np.ones((300, 300), bool)), 0.1)
    assert_within(o[:300], ref, tol)
    assert bool(torch.isnan(o[300:]).all())


def test_no_rows():
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    st = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    tgdn.prompt_attention(cu, e, e[:, :1], e[:, :1], e, 0.1, st)
    assert st.tolist() == [0, 0, 0]


def test_binding_refusals():
    cu, q, k, v = make([8], 4, 2, 64, BF)
    o, st = torch.empty_like(q), torch.empty(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        tgdn.prompt_attention(cu, q.transpose(1, 2).contiguous().transpose(1, 2), k, v, o, 0.1, st)
    with pytest.raises(TypeError):
        tgdn.prompt_attention(cu, q, k.half(), v, o, 0.1, st)
    with pytest.raises(ValueError, match="shape"):
        tgdn.prompt_attention(cu, q, k, v[:4], o, 0.1, st)
    with pytest.raises(TypeError):
        tgdn.prompt_attention(cu.long(), q, k, v, o, 0.1, st)
    with pytest.raises(tgdn.TgdnError) as e:
        tgdn.prompt_attention(cu, q, k, v, o, float("nan"), st)
    assert e.value.code == tgdn.EINVAL


def test_in_a_graph_and_on_a_side_stream():
    cu, q, k, v = make([300, 20], 4, 1, 128, BF, seed=15)
    want, _ = run(cu, q, k, v, 0.088)
    side = torch.cuda.Stream()
    o, st = torch.zeros_like(q), torch.zeros(2, dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tgdn.prompt_attention(cu, q, k, v, o, 0.088, st)
    side.synchronize()
    assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        tgdn.prompt_attention(cu, q, k, v, o, 0.088, st)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
