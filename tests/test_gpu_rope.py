"""tgdn_rope against the formula in 64 bits: both pairings, part of the head, every io type,
long-context scalings, far positions, tree and prompt positions, strided and in-place rows;
its transpose against the formula and against differences; rows outside every sequence."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
from attn_helpers import HALF, inv_freq, rotate  # noqa: E402
from tree_speculative_decoding_gated_gb300 import tgdn  # noqa: E402

I32 = dict(dtype=torch.int32, device="cuda")


def make(T, heads, d, dtype, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    full = torch.randn((T, heads + pad, d), generator=g).to(dtype).cuda()
    return full[:, :heads]


def check(x, y, pos, f, m, inter, sign=1.0):
    ref, mag = rotate(x, pos, f, m, inter, sign)
    tol = HALF[x.dtype] * ref.abs() + 2.0 ** -21 * mag
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half of fp16's smallest step
    d = (y.cpu().double() - ref).abs()
    assert not bool((d > tol).any()), float((d - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H_q,H_kv,d,rot", [
    (1, 1, 1, 8, 2), (5, 4, 1, 64, 64), (33, 16, 4, 128, 128), (7, 3, 3, 96, 32), (40, 8, 2, 128, 36),
    (9, 2, 1, 256, 250), (1300, 5, 1, 16, 8), (700, 24, 8, 80, 80)])
def test_values(T, H_q, H_kv, d, rot, inter, dtype):
    rng = np.random.default_rng(T + d)
    cuts = np.sort(rng.integers(0, T + 1, 4))
    cu = [0, *cuts.tolist(), T]                       # empty sequences among them
    base = rng.integers(0, 100000, len(cu) - 1)
    off = rng.integers(0, 40, T)
    freq, m = tgdn.rope_freqs(rot, 10000.0, "none")
    q, k = make(T, H_q, d, dtype, 1, pad=2), make(T, H_kv, d, dtype, 2)
    qo, ko = torch.full_like(q.contiguous(), 7.0), make(T, H_kv, d, dtype, 3, pad=1)
    tgdn.rope(q, k, qo, ko, freq, cu=torch.tensor(cu, **I32), base=torch.tensor(base, **I32),
              off=torch.tensor(off, **I32), interleaved=inter, mscale=m)
    pos = np.repeat(base, np.diff(cu)) + off
    f, _ = inv_freq(rot, 10000.0)
    check(q, qo, pos, f, 1.0, inter)
    check(k, ko, pos, f, 1.0, inter)


@pytest.mark.parametrize("scaling,factor", [("linear", 8.0), ("ntk", 4.0), ("yarn", 16.0)])
def test_scalings_at_far_positions(scaling, factor):
    """Positions up to 2^31 - 1: the phase is exact where an fp32 angle has lost every bit."""
    T, d = 64, 128
    rng = np.random.default_rng(3)
    off = np.concatenate([[0, 1, 2 ** 31 - 1, 2 ** 30], rng.integers(0, 2 ** 31 - 1, T - 4)])
    freq, m = tgdn.rope_freqs(d, 500000.0, scaling, factor, 8192)
    # the angle itself in integers: position times the table's fraction of a turn
    table = [int(x) % 2 ** 64 for x in freq.tolist()]
    turn = np.array([[(int(p) * t % 2 ** 64) / 2.0 ** 64 for t in table] for p in off])
    f, wm = inv_freq(d, 500000.0, scaling, factor, 8192)
    assert abs(m - wm) < 1e-6
    # the table's half step, times the position
    assert np.abs(np.remainder(turn - np.outer(off, f) / (2 * np.pi) + 0.5, 1) - 0.5).max() < 2.0 ** -20
    q = make(T, 2, d, torch.float32, 5)
    qo = torch.empty_like(q)
    tgdn.rope(q, None, qo, None, freq, cu=torch.tensor([0, T], **I32), off=torch.tensor(off, **I32),
              mscale=m)
    a = torch.as_tensor(2 * np.pi * turn)
    c, s = (torch.cos(a) * m)[:, None], (torch.sin(a) * m)[:, None]
    x = q.cpu().double()
    ref = torch.cat([x[..., :64] * c - x[..., 64:] * s, x[..., :64] * s + x[..., 64:] * c], -1)
    mag = (x[..., :64].abs() + x[..., 64:].abs()) * m
    tol = HALF[torch.float32] * ref.abs() + 2.0 ** -21 * torch.cat([mag, mag], -1)
    assert bool(((qo.cpu().double() - ref).abs() <= tol).all())


def test_positions_default_to_the_index_in_the_sequence():
    T, d = 50, 64
    freq, _ = tgdn.rope_freqs(d)
    q = make(T, 2, d, torch.bfloat16, 8)
    qo = torch.empty_like(q)
    tgdn.rope(q, None, qo, None, freq, cu=torch.tensor([0, 20, 20, 50], **I32))
    check(q, qo, np.r_[np.arange(20), np.arange(30)], inv_freq(d, 10000.0)[0], 1.0, False)


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_equals_out_of_place(inter):
    T, d = 70, 96
    freq, _ = tgdn.rope_freqs(64)
    qkv = make(T, 12, d, torch.bfloat16, 9)
    q, k = qkv[:, :8], qkv[:, 8:10]
    cu, base = torch.tensor([0, T], **I32), torch.tensor([300], **I32)
    qo, ko = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    tgdn.rope(q, k, qo, ko, freq, cu=cu, base=base, interleaved=inter)
    rest = qkv[:, 10:].clone()
    tgdn.rope(q, k, q, k, freq, cu=cu, base=base, interleaved=inter)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, 10:], rest)


@pytest.mark.parametrize("inter", [False, True])
def test_transpose_is_the_gradient(inter):
    """<y, R x> = <R^T y, x> by the formula, and R^T y against differences of <y, R x>."""
    T, d, rot = 6, 32, 24
    freq, m = tgdn.rope_freqs(rot, 10000.0, "yarn", 4.0, 16)
    cu, off = torch.tensor([0, T], **I32), torch.tensor([0, 3, 9, 1000, 65536, 7], **I32)
    f, _ = inv_freq(rot, 10000.0, "yarn", 4.0, 16)
    y = make(T, 2, d, torch.float32, 11)
    g = torch.empty_like(y)
    tgdn.rope(y, None, g, None, freq, cu=cu, off=off, interleaved=inter, mscale=m, transpose=True)
    check(y, g, off.cpu().numpy(), f, m, inter, sign=-1.0)
    x = make(T, 2, d, torch.float32, 12)
    out = torch.empty_like(x)

    def value(z):  # <y, R z> in fp64 over the kernel's fp32 outputs
        tgdn.rope(z, None, out, None, freq, cu=cu, off=off, interleaved=inter, mscale=m)
        return float((y.double() * out.double()).sum())

    rng = np.random.default_rng(0)
    for _ in range(12):
        t, h, i = rng.integers(T), rng.integers(2), rng.integers(d)
        e = torch.zeros_like(x)
        e[t, h, i] = 1.0   # the map is linear: a whole step is no approximation
        diff = value(x + e) - value(x - e)
        # each of the two sums rounds its changed pair: 2^-21 of |x| + 1 times |y|, twice
        assert abs(diff / 2 - float(g[t, h, i])) <= 2.0 ** -19 * (1 + float(x.abs().max())) * \
            float(y.abs().max()) * m


def test_rows_outside_the_sequences_are_left_alone():
    T, d = 12, 64
    freq, _ = tgdn.rope_freqs(d)
    q = make(T, 1, d, torch.bfloat16, 13)
    qo = torch.full_like(q, 5.0)
    tgdn.rope(q, None, qo, None, freq, cu=torch.tensor([2, 5, 8], **I32))
    assert bool((qo[:2] == 5).all()) and bool((qo[8:] == 5).all()) and bool((qo[3:5] != 5).any())
    qo.fill_(5.0)
    tgdn.rope(q, None, qo, None, freq, cu=torch.tensor([0, 4, 40], **I32))  # the second leaves [0, T)
    assert bool((qo[4:] == 5).all()) and bool((qo[1:4] != 5).any())


def test_non_finite_values_stay_in_their_pair():
    T, d = 3, 64
    freq, _ = tgdn.rope_freqs(d)
    q = make(T, 2, d, torch.bfloat16, 14)
    clean, got = torch.empty_like(q), torch.empty_like(q)
    cu = torch.tensor([0, T], **I32)
    tgdn.rope(q, None, clean, None, freq, cu=cu)
    bad = q.clone()
    bad[1, 1, 5] = float("nan")
    tgdn.rope(bad, None, got, None, freq, cu=cu)
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[1, 1, 5] = hit[1, 1, 37] = True
    assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], clean[~hit])


def test_decreasing_offsets_hide_no_sound_sequence():
    T, d = 20, 64
    freq, _ = tgdn.rope_freqs(d)
    q = make(T, 1, d, torch.bfloat16, 15)
    qo = torch.full_like(q, 5.0)
    tgdn.rope(q, None, qo, None, freq, cu=torch.tensor([0, 6, 3, 3, 90], **I32))
    check(q[:6], qo[:6], np.arange(6), inv_freq(d, 10000.0)[0], 1.0, False)
    assert bool((qo[6:] == 5).all())
