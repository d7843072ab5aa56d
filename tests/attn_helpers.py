"""Plain 64-bit statements of the attention-layer operators, and their tolerances.

Tolerances count roundings.  With u = eps / 2 of the io type (half a step, relative):
  * a probability enters the second product rounded to the io type: it is off by u p, and in
    fp16 (whose smallest step is 2^-24) by 2^-25 at least; the output is rounded once more:
        |o - o_ref| <= u (A + |o|) + 2^-25 V / l + 2^-12 A,   A = sum_j p_j |v_j|
    (V the sum of |v_j| over the visible keys, l >= 1 the kernel's sum of exponentials).
    The last term is for fp32 work: scores summed over d <= 128 terms in fp32 carry at most
    d 2^-23 of scale sum |q k| <= 16 here, and the base-2 exponential 2^-22.
  * a rotated value is off by u of itself and by the angle: half a step of an fp32 fraction of
    a half turn (2^-25 pi) and two units of the fp32 sine and cosine: under 2^-21 (|x| + |y|).
"""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def visible_tree(parent):
    """Boolean [N][N]: node n sees s when s is on n's root path."""
    N = len(parent)
    see = np.zeros((N, N), bool)
    for n in range(N):
        j = n
        while j != -1:
            see[n, j] = True
            j = int(parent[j])
    return see


def attend(q, k, v, see, scale):
    """q [n][H_q][d], k, v [m][H_kv][d], see [n][m]: (o, tolerance) in fp64, o zero where a row
    sees nothing."""
    u = HALF[q.dtype]
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    see = torch.as_tensor(np.asarray(see))
    G = q.shape[1] // k.shape[1]
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    for h in range(q.shape[1]):
        s = scale * q[:, h] @ k[:, h // G].T
        s = torch.where(see, s, torch.full_like(s, -math.inf))
        m = s.amax(1, keepdim=True)
        p = torch.where(see, torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m)),
                        torch.zeros_like(s))
        total = p.sum(1, keepdim=True)
        total[total == 0] = 1.0
        p = p / total
        vv = v[:, h // G]
        o[:, h] = p @ vv
        A = p @ vv.abs()
        V = see.double() @ vv.abs()
        tol[:, h] = u * (A + o[:, h].abs()) + 2.0 ** -25 * V + 2.0 ** -12 * A + 1e-30
    return o, tol


def assert_within(got, ref, tol, what=""):
    d = (got.detach().cpu().double() - ref).abs()
    assert bool(torch.isfinite(got.detach().cpu().double()).all()), what
    bad = d > tol
    assert not bool(bad.any()), (what, int(bad.sum()), float((d / tol).max()))
    return float((d / tol).max()) if d.numel() else 0.0


def inv_freq(rot, theta, scaling="none", factor=1.0, orig=0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, by the published formulas, and the value factor."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        pair = lambda t: rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(pair(beta_fast)), 0.0), min(math.ceil(pair(beta_slow)), rot - 1.0)
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * r + f * (1 - r), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, pos, f, mscale, interleaved, sign=1.0):
    """x [T][H][d] (any dtype), pos [T]: (y, |x| + |y| per pair) in fp64."""
    y = x.detach().cpu().double().clone()
    mag = torch.zeros_like(y)
    half = len(f)
    a = torch.as_tensor(np.outer(np.asarray(pos, np.float64), f)) * sign
    c, s = (torch.cos(a) * mscale)[:, None], (torch.sin(a) * mscale)[:, None]
    i0 = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    i1 = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    p, q = y[..., i0].clone(), y[..., i1].clone()
    y[..., i0], y[..., i1] = p * c - q * s, p * s + q * c
    mag[..., i0] = mag[..., i1] = (p.abs() + q.abs()) * mscale
    return y, mag
