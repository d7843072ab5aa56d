"""CPU checks of the attention-layer calls (rotary positions, prompt attention, paged cache,
paged tree attention): struct layouts, the frequency table against its formulas, and every
host-side refusal, before anything could be launched."""
import ctypes
import math

import numpy as np
import pytest

from tree_speculative_decoding_gated_gb300 import tgdn
from attn_helpers import inv_freq

FAKE = 0x10000  # a non-null, 256-byte aligned address; never dereferenced on the host


@pytest.fixture(scope="module")
def L():
    from tree_speculative_decoding_gated_gb300 import build
    build.build()
    return tgdn.lib()


def ctree(B=2, T=10, n_max=8, depth_max=4):
    return tgdn.CTree(B, T, n_max, depth_max, (n_max + 63) // 64, *([FAKE] * 7))


def cpages(B=2, n_pages=20, page_size=16, max_pages=8, **kw):
    f = dict(table=FAKE, len=FAKE, held=FAKE, refs=FAKE, status=FAKE, **kw)
    return tgdn.CPages(B, n_pages, page_size, max_pages, f["table"], f["len"], f["held"], f["refs"],
                       f["status"])


def cpool(layers=1, H_kv=2, d=64, data=FAKE):
    return tgdn.CPool(layers, H_kv, d, data)


def test_struct_layouts():
    assert ctypes.sizeof(tgdn.CPages) == 4 * 4 + 5 * 8 and tgdn.CPages.table.offset == 16
    assert ctypes.sizeof(tgdn.CPool) == 24 and tgdn.CPool.data.offset == 16


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("rot,theta,scaling,factor,orig", [
    (128, 10000.0, "none", 1.0, 0), (64, 1e6, "linear", 4.0, 0), (96, 10000.0, "ntk", 8.0, 0),
    (128, 10000.0, "yarn", 8.0, 4096), (64, 5e5, "yarn", 1.0, 8192), (2, 10000.0, "none", 1.0, 0),
    (4, 10000.0, "ntk", 2.0, 0), (32, 10000.0, "yarn", 16.0, 2), (256, 10.0, "yarn", 3.0, 100000)])
def test_frequencies(L, rot, theta, scaling, factor, orig):
    freq, m = tgdn.rope_freqs(rot, theta, scaling, factor, orig, device="cpu")
    want, wm = inv_freq(rot, theta, scaling, factor, orig)
    # fractions of a turn in steps of 2^-64: half a step, and the roundings of the power and of
    # the divisions in fp64
    got = [int(x) % 2 ** 64 for x in freq.tolist()]
    for g, w in zip(got, want / (2 * math.pi) * 2.0 ** 64):
        assert abs(g - w) <= 0.5 + 2.0 ** -48 * w, (g, w)
    assert abs(m - wm) <= 2.0 ** -23 * wm


def test_frequency_refusals(L):
    out, ms = (ctypes.c_uint64 * 128)(), ctypes.c_float()

    def call(rot=64, theta=1e4, scaling=0, factor=1.0, orig=4096, fast=32.0, slow=1.0, f=out, m=ms):
        return L.tgdn_rope_freqs(rot, theta, scaling, factor, orig, fast, slow, f,
                                 None if m is None else ctypes.byref(m))

    assert call() == tgdn.OK
    for kw in (dict(rot=0), dict(rot=63), dict(theta=1.0), dict(theta=math.nan), dict(theta=math.inf),
               dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5),
               dict(scaling=2, factor=math.inf), dict(scaling=2, rot=2, factor=2.0),
               dict(scaling=3, factor=2.0, orig=0), dict(scaling=3, factor=2.0, slow=0.0),
               dict(scaling=3, factor=2.0, fast=1.0, slow=1.0), dict(f=None), dict(m=None)):
        assert call(**kw) == tgdn.EINVAL, kw
    assert call(rot=258) == tgdn.ETOOBIG
    with pytest.raises(ValueError, match="scaling"):
        tgdn.rope_freqs(64, scaling="cubic", device="cpu")


def test_rope_refusals(L):
    def call(B=1, T=4, H_q=2, H_kv=1, d=64, rot=64, inter=0, tr=0, io=tgdn.BF16, m=1.0, freq=FAKE,
             cu=FAKE, q=FAKE, qs=128, k=FAKE * 2, ks=64, qo=FAKE * 3, qos=128, ko=FAKE * 4, kos=64):
        return L.tgdn_rope(B, T, H_q, H_kv, d, rot, inter, tr, io, m, freq, cu, None, None, q, qs, k,
                           ks, qo, qos, ko, kos, None)

    for kw in (dict(B=-1), dict(T=-1), dict(H_q=0), dict(H_kv=-1), dict(d=60), dict(d=0), dict(rot=0),
               dict(rot=33), dict(rot=66), dict(io=3), dict(m=math.nan), dict(freq=None),
               dict(cu=None), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None),
               dict(q=FAKE + 8), dict(qs=120), dict(qs=132), dict(ks=60), dict(ko=FAKE * 4 + 2),
               dict(qos=64), dict(qo=FAKE, qos=136), dict(ko=FAKE * 2, kos=72)):
        assert call(**kw) == tgdn.EINVAL, kw
    assert call(d=264, rot=8) == tgdn.ETOOBIG
    assert call(B=0, cu=None) == tgdn.OK and call(T=0, q=None) == tgdn.OK


# ------------------------------------------------------------------ prompt attention
def test_prompt_attention_refusals(L):
    def call(B=1, T=4, H_q=4, H_kv=2, d=64, io=tgdn.BF16, cu=FAKE, q=FAKE, qs=256, k=FAKE, ks=128,
             v=FAKE, vs=128, scale=0.1, o=FAKE, os=256, status=FAKE):
        return L.tgdn_prompt_attention(B, T, H_q, H_kv, d, io, cu, q, qs, k, ks, v, vs, scale, o, os,
                                       status, None, 0, None)

    for kw in (dict(B=-1), dict(T=-1), dict(H_q=0), dict(H_kv=0), dict(H_q=3), dict(d=0), dict(cu=None),
               dict(status=None), dict(q=None), dict(k=None), dict(v=None), dict(o=None),
               dict(q=FAKE + 2), dict(o=FAKE + 8), dict(qs=255), dict(qs=248), dict(ks=120),
               dict(vs=64), dict(os=128), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
               dict(scale=math.inf)):
        assert call(**kw) == tgdn.EINVAL, kw
    for kw in (dict(d=60, qs=240, ks=120, vs=120, os=240), dict(io=tgdn.F32),
               dict(H_q=258, H_kv=2, qs=258 * 64, os=258 * 64)):
        assert call(**kw) == tgdn.EUNSUPPORTED, kw
    assert call(d=136, qs=1024, ks=1024, vs=1024, os=1024) == tgdn.ETOOBIG
    assert call(B=0, cu=None, status=None) == tgdn.OK
    assert L.tgdn_prompt_attention_workspace_bytes(1, 4, 4, 2, 64) == 0


# ------------------------------------------------------------------ paged cache
BAD_PAGES = [dict(B=-1), dict(n_pages=-1), dict(max_pages=-1), dict(page_size=8), dict(page_size=48),
             dict(page_size=512), dict(table=None), dict(len=None), dict(held=None), dict(refs=None),
             dict(status=None)]


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_every_page_call_refuses_a_bad_cache(L, kw):
    args = {k: v for k, v in kw.items() if k in ("B", "n_pages", "page_size", "max_pages")}
    p = cpages(**args)
    for k, v in kw.items():
        if k not in args:
            setattr(p, k, v)
    P, pool, t = ctypes.byref(p), cpool(), ctree()
    assert L.tgdn_pages_reserve(P, FAKE, FAKE, None) == tgdn.EINVAL
    assert L.tgdn_pages_append(P, ctypes.byref(pool), 4, FAKE, None, 0, None, FAKE, 0, 128, FAKE, 0,
                               128, 1, None) == tgdn.EINVAL
    assert L.tgdn_pages_fork(P, ctypes.byref(pool), 1, FAKE, FAKE, FAKE, FAKE, None) == tgdn.EINVAL
    assert L.tgdn_pages_free(P, 1, FAKE, None) == tgdn.EINVAL
    assert L.tgdn_pages_compact(P, ctypes.byref(pool), FAKE, FAKE, None) == tgdn.EINVAL
    assert L.tgdn_pages_workspace_bytes(P) == 0
    assert L.tgdn_paged_tree_attention(ctypes.byref(t), P, 4, 2, 64, tgdn.BF16, FAKE, 256, FAKE, 128,
                                       FAKE, 128, FAKE, FAKE, 0.1, FAKE, 256, None, 0,
                                       None) == tgdn.EINVAL


def test_page_call_refusals(L):
    p, pool = cpages(), cpool()
    P, Q = ctypes.byref(p), ctypes.byref(pool)
    assert L.tgdn_pages_workspace_bytes(P) > 0
    assert L.tgdn_pages_reserve(P, None, FAKE, None) == tgdn.EINVAL
    assert L.tgdn_pages_reserve(P, FAKE, None, None) == tgdn.EINVAL
    assert L.tgdn_pages_reserve(P, FAKE, FAKE + 16, None) == tgdn.EINVAL
    assert L.tgdn_pages_reserve(None, FAKE, FAKE, None) == tgdn.EINVAL

    def append(pool=pool, T=4, cu=FAKE, path=None, plen=0, n=None, k=FAKE, kl=0, kr=128, v=FAKE, vl=0,
               vr=128):
        return L.tgdn_pages_append(P, ctypes.byref(pool), T, cu, path, plen, n, k, kl, kr, v, vl, vr, 1,
                                   None)

    for kw in (dict(T=-1), dict(cu=None), dict(path=FAKE, plen=4), dict(path=FAKE, plen=-1, n=FAKE),
               dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(kr=120), dict(vr=130),
               dict(pool=cpool(layers=0)), dict(pool=cpool(H_kv=0)), dict(pool=cpool(d=60)),
               dict(pool=cpool(d=0)), dict(pool=cpool(data=None)), dict(pool=cpool(data=FAKE + 8)),
               dict(pool=cpool(layers=2), kl=4), dict(pool=cpool(layers=2), vl=-8)):
        assert append(**kw) == tgdn.EINVAL, kw
    assert append(pool=cpool(d=264)) == tgdn.ETOOBIG
    assert append(pool=cpool(layers=40000)) == tgdn.ETOOBIG

    def fork(n=1, src=FAKE, dst=FAKE, st=FAKE, ws=FAKE):
        return L.tgdn_pages_fork(P, Q, n, src, dst, st, ws, None)

    for kw in (dict(n=-1), dict(src=None), dict(dst=None), dict(st=None), dict(ws=None),
               dict(ws=FAKE + 128)):
        assert fork(**kw) == tgdn.EINVAL, kw
    assert fork(n=4097) == tgdn.ETOOBIG
    assert fork(n=0, src=None) == tgdn.OK
    assert L.tgdn_pages_free(P, -1, FAKE, None) == tgdn.EINVAL
    assert L.tgdn_pages_free(P, 1, None, None) == tgdn.EINVAL
    assert L.tgdn_pages_free(P, 0, None, None) == tgdn.OK
    assert L.tgdn_pages_compact(P, Q, None, FAKE, None) == tgdn.EINVAL
    assert L.tgdn_pages_compact(P, Q, FAKE, None, None) == tgdn.EINVAL
    big = cpages(n_pages=(1 << 28) + 1)
    assert L.tgdn_pages_reserve(ctypes.byref(big), FAKE, FAKE, None) == tgdn.ETOOBIG
    empty = cpages(B=0)
    assert L.tgdn_pages_reserve(ctypes.byref(empty), None, None, None) == tgdn.OK


# ------------------------------------------------------------------ paged tree attention
def test_paged_tree_attention_refusals(L):
    def call(tree=None, pages=None, H_q=4, H_kv=2, d=64, io=tgdn.BF16, q=FAKE, qs=256, k=FAKE, ks=128,
             v=FAKE, vs=128, kp=FAKE, vp=FAKE, scale=0.1, o=FAKE, os=256, ws=None, wsn=0):
        t, p = tree or ctree(), pages or cpages()
        return L.tgdn_paged_tree_attention(ctypes.byref(t), ctypes.byref(p), H_q, H_kv, d, io, q, qs, k,
                                           ks, v, vs, kp, vp, scale, o, os, ws, wsn, None)

    for kw in (dict(tree=ctree(B=-1)), dict(tree=ctree(B=3)), dict(H_q=5), dict(H_kv=0), dict(d=0),
               dict(scale=0.0), dict(scale=math.nan), dict(q=None), dict(k=None), dict(v=None),
               dict(o=None), dict(kp=None), dict(vp=None), dict(kp=FAKE + 8), dict(q=FAKE + 2),
               dict(qs=250), dict(ks=64), dict(os=8), dict(ws=FAKE + 16)):
        assert call(**kw) == tgdn.EINVAL, kw
    assert call(io=tgdn.F32) == tgdn.EUNSUPPORTED
    assert call(d=36, qs=144, ks=72, vs=72, os=144) == tgdn.EUNSUPPORTED
    assert call(d=256, qs=1024, ks=512, vs=512, os=1024) == tgdn.ETOOBIG
    assert call(tree=ctree(n_max=257)) == tgdn.ETOOBIG
    assert L.tgdn_paged_tree_attention(None, ctypes.byref(cpages()), 4, 2, 64, 1, FAKE, 256, FAKE, 128,
                                       FAKE, 128, FAKE, FAKE, 0.1, FAKE, 256, None, 0,
                                       None) == tgdn.EINVAL
    t = ctree()
    assert L.tgdn_paged_tree_attention_workspace_bytes(ctypes.byref(t), 4, 2, 64) > 0
    assert L.tgdn_paged_tree_attention_workspace_bytes(ctypes.byref(t), 5, 2, 64) == 0


def test_f16_is_not_a_gdn_type(L):
    t, d = ctree(), tgdn.CDims(2, 4, 64, 64, tgdn.F16)
    assert L.tgdn_verify(ctypes.byref(t), ctypes.byref(d), *([FAKE] * 8), None) == tgdn.EINVAL


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    freq, _ = tgdn.rope_freqs(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        tgdn.rope(q, None, q, None, freq, cu=cu)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tgdn.prompt_attention(cu, q, q, q, q, 0.1, cu)
    with pytest.raises(TypeError):
        tgdn.prompt_attention(cu, q.to(torch.float64), q, q, q, 0.1, cu)
    pages = tgdn.Pages(2, 4, 16, 2, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        tgdn.pages_free(pages, cu)
    with pytest.raises(TypeError, match="pool"):
        tgdn._pool(pages, torch.zeros(1, 2, 4, 1, 16, 64))
    with pytest.raises(ValueError, match="pool"):
        tgdn._pool(pages, torch.zeros(1, 2, 5, 1, 16, 64, dtype=torch.float16))


def test_a_handle_sees_new_and_moved_tensors():
    """The kept C struct of a tree or cache is made (and checked) anew when an attribute is set
    or a tensor's storage moves."""
    torch = pytest.importorskip("torch")
    made = []

    class Counted(tgdn.Pages):
        def _make(self):
            made.append(1)
            return object()

    pages = Counted(2, 4, 16, 2, device="cpu")
    a = pages.c()
    assert pages.c() is a and len(made) == 1
    pages.len = torch.zeros(2, dtype=torch.int32)
    assert pages.c() is not a and len(made) == 2
    pages.refs.resize_(1 << 20)
    pages.c()
    assert len(made) == 3
