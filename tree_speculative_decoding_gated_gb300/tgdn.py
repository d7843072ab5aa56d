"""Thin Python binding of libtgdn.so (include/tgdn.h) — argument marshalling only.

Every step of the path runs in the library's CUDA kernels; this module only
checks that the torch tensors it is handed live on the GPU with the dtype,
layout and size the C ABI expects (a host pointer handed to a kernel would
fault the device), packs the C structs and raises on a non-zero status.  There
is no fallback: if the library has not been built this module fails to load.

Names follow the C ABI: tree_prep, verify_workspace_bytes, verify, accept,
commit.  All calls are asynchronous on the given stream (default: torch's
current stream).
"""
from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtgdn.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "tgdn.h")

OK, EINVAL, ETOOBIG, ECUDA, EUNSUPPORTED = 0, -1, -3, -4, -5
SEQ_OK, SEQ_TOO_BIG, SEQ_BAD_PARENT, SEQ_ROOTS, SEQ_CYCLE, SEQ_TOO_DEEP, SEQ_TIMEOUT = range(7)
SEQ_BAD_RANGE, SEQ_BAD_PAGE, SEQ_NO_PAGES = 7, 8, 9
F32, BF16, F16 = 0, 1, 2
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
MAX_NODES, MAX_DEPTH, MAX_HEAD_DIM = 256, 64, 128
NOALLOC_SCRATCH_BYTES = 20 * 1024 * 1024


class TgdnError(RuntimeError):
    def __init__(self, code: int, call: str):
        self.code = code
        super().__init__(f"{call}: {status_string(code)} ({code})")


class CTree(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("n_max", ctypes.c_int32),
                ("depth_max", ctypes.c_int32), ("words", ctypes.c_int32),
                ("cu_nodes", ctypes.c_void_p), ("parent", ctypes.c_void_p),
                ("depth", ctypes.c_void_p), ("order", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("anc", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class CDims(ctypes.Structure):
    _fields_ = [("H_qk", ctypes.c_int32), ("H_v", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("io", ctypes.c_int32)]


class CPages(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("table", ctypes.c_void_p),
                ("len", ctypes.c_void_p), ("held", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class CPool(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("data", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libtgdn.so; raises if it has not been built (there is no other path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
        P = ctypes.POINTER
        L.tgdn_tree_prep.argtypes = [P(CTree), st]
        L.tgdn_verify_workspace_bytes.argtypes = [P(CTree), P(CDims)]
        L.tgdn_verify_workspace_bytes.restype = ctypes.c_size_t
        L.tgdn_verify.argtypes = [P(CTree), P(CDims), vp, vp, vp, vp, vp, vp, vp, vp, st]
        L.tgdn_accept.argtypes = [P(CTree), vp, vp, vp, vp, vp, st]
        L.tgdn_commit.argtypes = [P(CTree), P(CDims), vp, vp, vp, vp, vp, st]
        L.tgdn_verify_recurrent.argtypes = [P(CTree), P(CDims), vp, vp, vp, vp, vp, vp, vp, st]
        L.tgdn_verify_recurrent.restype = ctypes.c_int
        L.tgdn_verify_noalloc.argtypes = [P(CTree), P(CDims), vp, vp, vp, vp, vp, vp, vp, st]
        L.tgdn_verify_noalloc.restype = ctypes.c_int
        L.tgdn_verify_fused.argtypes = [P(CTree), P(CDims), vp, vp, vp, vp, vp, vp, vp, vp,
                                        P(CTree), vp, vp, vp, vp, st]
        L.tgdn_verify_fused.restype = ctypes.c_int
        L.tgdn_tree_build.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                      vp, st]
        L.tgdn_tree_build.restype = ctypes.c_int
        L.tgdn_tree_attention.argtypes = [P(CTree), i32, i32, i32, vp, vp, vp, vp, vp, vp, i32,
                                          ctypes.c_float, vp, vp, ctypes.c_size_t, st]
        L.tgdn_tree_attention.restype = ctypes.c_int
        L.tgdn_tree_attention_workspace_bytes.argtypes = [P(CTree), i32, i32, i32, i32]
        L.tgdn_tree_attention_workspace_bytes.restype = ctypes.c_size_t
        L.tgdn_debug_set_wait_hooks.argtypes = [ctypes.c_uint64, ctypes.c_int32]
        L.tgdn_debug_set_wait_hooks.restype = ctypes.c_int
        i64, f32, f64, size = ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
        L.tgdn_rope_freqs.argtypes = [i32, f64, i32, f64, i32, f64, f64, vp, vp]
        L.tgdn_rope.argtypes = [i32] * 9 + [f32, vp, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, i64,
                                            st]
        L.tgdn_prompt_attention.argtypes = [i32] * 6 + [vp, vp, i64, vp, i64, vp, i64, f32, vp, i64,
                                                        vp, vp, size, st]
        L.tgdn_prompt_attention_workspace_bytes.argtypes = [i32] * 5
        L.tgdn_prompt_attention_workspace_bytes.restype = size
        L.tgdn_pages_workspace_bytes.argtypes = [P(CPages)]
        L.tgdn_pages_workspace_bytes.restype = size
        L.tgdn_pages_reserve.argtypes = [P(CPages), vp, vp, st]
        L.tgdn_pages_append.argtypes = [P(CPages), P(CPool), i32, vp, vp, i32, vp, vp, i64, i64, vp,
                                        i64, i64, i32, st]
        L.tgdn_pages_fork.argtypes = [P(CPages), P(CPool), i32, vp, vp, vp, vp, st]
        L.tgdn_pages_free.argtypes = [P(CPages), i32, vp, st]
        L.tgdn_pages_compact.argtypes = [P(CPages), P(CPool), vp, vp, st]
        L.tgdn_paged_tree_attention.argtypes = [P(CTree), P(CPages), i32, i32, i32, i32, vp, i64, vp,
                                                i64, vp, i64, vp, vp, f32, vp, i64, vp, size, st]
        L.tgdn_paged_tree_attention_workspace_bytes.argtypes = [P(CTree), i32, i32, i32]
        L.tgdn_paged_tree_attention_workspace_bytes.restype = size
        for f in (L.tgdn_rope_freqs, L.tgdn_rope, L.tgdn_prompt_attention, L.tgdn_pages_reserve,
                  L.tgdn_pages_append, L.tgdn_pages_fork, L.tgdn_pages_free, L.tgdn_pages_compact,
                  L.tgdn_paged_tree_attention):
            f.restype = ctypes.c_int
        L.tgdn_status_string.argtypes = [i32]
        L.tgdn_status_string.restype = ctypes.c_char_p
        L.tgdn_version.argtypes = []
        for f in (L.tgdn_tree_prep, L.tgdn_verify, L.tgdn_accept, L.tgdn_commit, L.tgdn_version):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


_calls = None


def _native():
    """The attention-layer calls' tensor marshalling in C++ (csrc/binding.cpp)."""
    global _calls
    if _calls is None:
        lib()
        try:
            from . import _calls as module
        except ImportError as e:
            raise RuntimeError("_calls.so is missing or does not load: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        _calls = module
    return _calls


def header_functions() -> list[str]:
    """Names of the functions include/tgdn.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]+?\b(tgdn_\w+)\s*\(", text, re.M)))


def status_string(code: int) -> str:
    return lib().tgdn_status_string(int(code)).decode()


def _check(rc: int, call: str):
    if rc != OK:
        raise TgdnError(rc, call)


# the handle of a device's current stream without a torch.cuda.Stream around it (about 3 us
# less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_get_device = getattr(torch._C, "_cuda_getDevice", None)
_Tensor = torch.Tensor


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_get_device() if _get_device is not None and
                               torch.cuda.is_initialized() else torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype, numel: int, name: str) -> int:
    """Device pointer of a contiguous CUDA tensor holding at least `numel` elements."""
    if isinstance(t, _Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous() and \
            t.numel() >= numel:
        return t.data_ptr() or None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (the library takes device pointers)")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: {t.numel()} elements, need {numel}")


@dataclass
class Dims:
    H_qk: int
    H_v: int
    d_k: int
    d_v: int
    io: int = BF16

    def c(self) -> CDims:
        return CDims(self.H_qk, self.H_v, self.d_k, self.d_v, self.io)

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.io == BF16 else torch.float32


class _Handle:
    """Device tensors behind a C struct.  The struct is made (and every tensor checked) again
    whenever an attribute is set or anything that the checks look at has changed: a tensor's
    address, place, type, size or contiguity."""

    _tensors: tuple = ()

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_struct"] = None

    def c(self):
        d = self.__dict__
        seen = []
        for n in self._tensors:
            t = d[n]
            seen += t.data_ptr(), t.is_cuda, t.dtype, t.numel(), t.is_contiguous()
        if d["_struct"] is None or d["_seen"] != seen:
            d["_struct"] = self._make()
            d["_seen"] = seen
        return d["_struct"]


class Tree(_Handle):
    """A batch of draft trees on the device plus the metadata tree_prep writes."""

    _tensors = ("cu_nodes", "parent", "depth", "order", "pos", "anc", "status")

    def __init__(self, cu_nodes: torch.Tensor, parent: torch.Tensor, n_max: int,
                 depth_max: int, T: int | None = None):
        self.B = int(cu_nodes.numel()) - 1
        self.T = int(parent.numel()) if T is None else int(T)
        self.n_max, self.depth_max = int(n_max), int(depth_max)
        self.words = max(1, (self.n_max + 63) // 64)
        dev = cu_nodes.device
        self.cu_nodes, self.parent = cu_nodes, parent
        self.depth = torch.empty(self.T, dtype=torch.int32, device=dev)
        self.order = torch.empty(self.T, dtype=torch.int32, device=dev)
        self.pos = torch.empty(self.T, dtype=torch.int32, device=dev)
        self.anc = torch.empty((self.T, self.words), dtype=torch.int64, device=dev)
        self.status = torch.empty(max(self.B, 0), dtype=torch.int32, device=dev)

    @classmethod
    def from_host(cls, cu_nodes, parent, n_max: int, depth_max: int, device="cuda"):
        cu = torch.as_tensor(cu_nodes, dtype=torch.int32).to(device)
        par = torch.as_tensor(parent, dtype=torch.int32).to(device)
        return cls(cu, par, n_max, depth_max)

    def _make(self) -> CTree:
        B, T = self.B, self.T
        return CTree(B, T, self.n_max, self.depth_max, self.words,
                     _dev(self.cu_nodes, torch.int32, B + 1, "cu_nodes"),
                     _dev(self.parent, torch.int32, T, "parent"),
                     _dev(self.depth, torch.int32, T, "depth"),
                     _dev(self.order, torch.int32, T, "order"),
                     _dev(self.pos, torch.int32, T, "pos"),
                     _dev(self.anc, torch.int64, T * self.words, "anc"),
                     _dev(self.status, torch.int32, B, "status"))


def tree_prep(tree: Tree, stream=None) -> None:
    ct = tree.c()
    _check(lib().tgdn_tree_prep(ctypes.byref(ct), _stream(stream)), "tgdn_tree_prep")


def verify_workspace_bytes(tree: Tree, dims: Dims) -> int:
    ct, cd = tree.c(), dims.c()
    return int(lib().tgdn_verify_workspace_bytes(ctypes.byref(ct), ctypes.byref(cd)))


def alloc_workspace(tree: Tree, dims: Dims, device="cuda") -> torch.Tensor:
    n = verify_workspace_bytes(tree, dims)
    if n == 0 and tree.T > 0:
        raise TgdnError(EINVAL, "tgdn_verify_workspace_bytes")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def verify(tree: Tree, dims: Dims, q, k, v, g, b, S0, o, ws, stream=None) -> None:
    T, B = tree.T, tree.B
    io = dims.torch_dtype
    ct, cd = tree.c(), dims.c()
    args = (_dev(q, io, T * dims.H_qk * dims.d_k, "q"), _dev(k, io, T * dims.H_qk * dims.d_k, "k"),
            _dev(v, io, T * dims.H_v * dims.d_v, "v"), _dev(g, torch.float32, T * dims.H_v, "g"),
            _dev(b, torch.float32, T * dims.H_v, "b"),
            _dev(S0, torch.float32, B * dims.H_v * dims.d_k * dims.d_v, "S0"),
            _dev(o, io, T * dims.H_v * dims.d_v, "o"),
            _dev(ws, torch.uint8, verify_workspace_bytes(tree, dims), "ws"))
    _check(lib().tgdn_verify(ctypes.byref(ct), ctypes.byref(cd), *args, _stream(stream)),
           "tgdn_verify")


def verify_fused(tree: Tree, dims: Dims, q, k, v, g, b, S, o, ws, prev_tree: Tree,
                 prev_accept_node, prev_path, prev_k, prev_ws, stream=None) -> None:
    """tgdn_verify_fused: commit the previous step's accepted node into S (in place),
    then verify this step's tree from the committed state."""
    T, B = tree.T, tree.B
    io = dims.torch_dtype
    ct, cd, pt = tree.c(), dims.c(), prev_tree.c()
    args = (_dev(q, io, T * dims.H_qk * dims.d_k, "q"), _dev(k, io, T * dims.H_qk * dims.d_k, "k"),
            _dev(v, io, T * dims.H_v * dims.d_v, "v"), _dev(g, torch.float32, T * dims.H_v, "g"),
            _dev(b, torch.float32, T * dims.H_v, "b"),
            _dev(S, torch.float32, B * dims.H_v * dims.d_k * dims.d_v, "S"),
            _dev(o, io, T * dims.H_v * dims.d_v, "o"),
            _dev(ws, torch.uint8, verify_workspace_bytes(tree, dims), "ws"))
    prev = (_dev(prev_accept_node, torch.int32, prev_tree.B, "prev_accept_node"),
            _dev(prev_path, torch.int32, prev_tree.B * (prev_tree.depth_max + 1), "prev_path"),
            _dev(prev_k, io, prev_tree.T * dims.H_qk * dims.d_k, "prev_k"),
            _dev(prev_ws, torch.uint8, verify_workspace_bytes(prev_tree, dims), "prev_ws"))
    _check(lib().tgdn_verify_fused(ctypes.byref(ct), ctypes.byref(cd), *args, ctypes.byref(pt),
                                   *prev, _stream(stream)), "tgdn_verify_fused")


def verify_recurrent(tree: Tree, dims: Dims, q, k, v, g, b, S0, o, stream=None) -> None:
    """tgdn_verify_recurrent: the per-branch recurrent baseline (same outputs as verify)."""
    T, B = tree.T, tree.B
    io = dims.torch_dtype
    ct, cd = tree.c(), dims.c()
    args = (_dev(q, io, T * dims.H_qk * dims.d_k, "q"), _dev(k, io, T * dims.H_qk * dims.d_k, "k"),
            _dev(v, io, T * dims.H_v * dims.d_v, "v"), _dev(g, torch.float32, T * dims.H_v, "g"),
            _dev(b, torch.float32, T * dims.H_v, "b"),
            _dev(S0, torch.float32, B * dims.H_v * dims.d_k * dims.d_v, "S0"),
            _dev(o, io, T * dims.H_v * dims.d_v, "o"))
    _check(lib().tgdn_verify_recurrent(ctypes.byref(ct), ctypes.byref(cd), *args,
                                       _stream(stream)), "tgdn_verify_recurrent")


BUILD_MAX_K = 16


def tree_build(root_token, child_logp, child_token, budget: int, w: int, depth_max: int,
               out=None, stream=None) -> dict:
    """tgdn_tree_build: top-w best-first draft trees for a batch of sequences.
    root_token [B] int32, child_logp [B][budget][K] fp32, child_token [B][budget][K] int32.
    Returns (or fills `out` with) parent/token/depth [B][budget] int32, score [B][budget]
    fp32, n_nodes [B] and rounds [B] int32, all on the device."""
    B = root_token.shape[0]
    K = child_logp.shape[-1] if child_logp.dim() == 3 else 0
    dev = root_token.device
    if out is None:
        out = dict(parent=torch.empty((B, budget), dtype=torch.int32, device=dev),
                   token=torch.empty((B, budget), dtype=torch.int32, device=dev),
                   score=torch.empty((B, budget), dtype=torch.float32, device=dev),
                   depth=torch.empty((B, budget), dtype=torch.int32, device=dev),
                   n_nodes=torch.empty(B, dtype=torch.int32, device=dev),
                   rounds=torch.empty(B, dtype=torch.int32, device=dev))
    nt = B * budget * K
    args = (_dev(root_token, torch.int32, B, "root_token"),
            _dev(child_logp, torch.float32, nt, "child_logp"),
            _dev(child_token, torch.int32, nt, "child_token"),
            _dev(out["parent"], torch.int32, B * budget, "parent"),
            _dev(out["token"], torch.int32, B * budget, "token"),
            _dev(out["score"], torch.float32, B * budget, "score"),
            _dev(out["depth"], torch.int32, B * budget, "depth"),
            _dev(out["n_nodes"], torch.int32, B, "n_nodes"),
            _dev(out["rounds"], torch.int32, B, "rounds"))
    _check(lib().tgdn_tree_build(B, budget, K, w, depth_max, *args, _stream(stream)),
           "tgdn_tree_build")
    return out


def tree_attention_workspace_bytes(tree: Tree, H_q: int, H_kv: int, d: int, P_max: int) -> int:
    return int(lib().tgdn_tree_attention_workspace_bytes(ctypes.byref(tree.c()), H_q, H_kv, d,
                                                         P_max))


def tree_attention(tree: Tree, q, k_tree, v_tree, k_cache, v_cache, prefix_len, o,
                   scale: float, ws=None, stream=None) -> None:
    """tgdn_tree_attention: each node attends to its sequence's cached context and its
    own root path.  q/o [T][H_q][d], k_tree/v_tree [T][H_kv][d], k_cache/v_cache
    [B][P_max][H_kv][d] (bf16), prefix_len [B] int32; scale positive and finite (the
    logits are scale * q.k).  ws: optional uint8 workspace of
    tree_attention_workspace_bytes() bytes (splits the cached context over more CTAs)."""
    T, B = tree.T, tree.B
    H_q, d = q.shape[1], q.shape[2]
    H_kv = k_tree.shape[1]
    P_max = k_cache.shape[1] if k_cache is not None else 0
    bf = torch.bfloat16
    ncache = B * P_max * H_kv * d
    args = (_dev(q, bf, T * H_q * d, "q"), _dev(k_tree, bf, T * H_kv * d, "k_tree"),
            _dev(v_tree, bf, T * H_kv * d, "v_tree"),
            _dev(k_cache, bf, ncache, "k_cache") if P_max > 0 else None,
            _dev(v_cache, bf, ncache, "v_cache") if P_max > 0 else None,
            _dev(prefix_len, torch.int32, B, "prefix_len"))
    wsp, wsn = None, 0
    if ws is not None:
        wsn = ws.numel() * ws.element_size()
        wsp = _dev(ws, ws.dtype, ws.numel(), "ws") if wsn > 0 else None
    _check(lib().tgdn_tree_attention(ctypes.byref(tree.c()), H_q, H_kv, d, *args, P_max,
                                     float(scale), _dev(o, bf, T * H_q * d, "o"), wsp, wsn,
                                     _stream(stream)), "tgdn_tree_attention")


def accept(tree: Tree, draft_ids, target_ids, accept_node, accept_len, path, stream=None) -> None:
    T, B = tree.T, tree.B
    ct = tree.c()
    args = (_dev(draft_ids, torch.int32, T, "draft_ids"),
            _dev(target_ids, torch.int32, T, "target_ids"),
            _dev(accept_node, torch.int32, B, "accept_node"),
            _dev(accept_len, torch.int32, B, "accept_len"),
            _dev(path, torch.int32, B * (tree.depth_max + 1), "path"))
    _check(lib().tgdn_accept(ctypes.byref(ct), *args, _stream(stream)), "tgdn_accept")


def commit(tree: Tree, dims: Dims, accept_node, k, ws, S_in, S_out, stream=None) -> None:
    T, B = tree.T, tree.B
    ct, cd = tree.c(), dims.c()
    ns = B * dims.H_v * dims.d_k * dims.d_v
    args = (_dev(accept_node, torch.int32, B, "accept_node"),
            _dev(k, dims.torch_dtype, T * dims.H_qk * dims.d_k, "k"),
            _dev(ws, torch.uint8, verify_workspace_bytes(tree, dims), "ws"),
            _dev(S_in, torch.float32, ns, "S_in"), _dev(S_out, torch.float32, ns, "S_out"))
    _check(lib().tgdn_commit(ctypes.byref(ct), ctypes.byref(cd), *args, _stream(stream)),
           "tgdn_commit")


def verify_noalloc(tree: Tree, dims: Dims, q, k, v, g, b, S0, o, stream=None) -> None:
    """tgdn_verify_noalloc: verification for callers that cannot allocate device memory.

    Same outputs as verify(); the factors stay in a library-owned device array of
    NOALLOC_SCRATCH_BYTES (so they cannot be committed from).  Calls on one device share
    that array: keep them ordered on one stream."""
    T, B = tree.T, tree.B
    io = dims.torch_dtype
    ct, cd = tree.c(), dims.c()
    args = (_dev(q, io, T * dims.H_qk * dims.d_k, "q"), _dev(k, io, T * dims.H_qk * dims.d_k, "k"),
            _dev(v, io, T * dims.H_v * dims.d_v, "v"), _dev(g, torch.float32, T * dims.H_v, "g"),
            _dev(b, torch.float32, T * dims.H_v, "b"),
            _dev(S0, torch.float32, B * dims.H_v * dims.d_k * dims.d_v, "S0"),
            _dev(o, io, T * dims.H_v * dims.d_v, "o"))
    _check(lib().tgdn_verify_noalloc(ctypes.byref(ct), ctypes.byref(cd), *args, _stream(stream)),
           "tgdn_verify_noalloc")


# ---------------------------------------------------------------- attention layers
def rope_freqs(rot: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               orig_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """tgdn_rope_freqs: (freq, mscale) for rope().  freq [rot / 2] on `device`: each pair's turns
    per position as 64-bit fractions (int64 storage); scaling "none", "linear", "ntk" or "yarn"."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling: {scaling!r}, expected one of {sorted(ROPE_SCALING)}")
    freq = torch.empty(max(rot // 2, 1), dtype=torch.int64)
    mscale = ctypes.c_float()
    _check(lib().tgdn_rope_freqs(rot, theta, ROPE_SCALING[scaling], factor, orig_len, beta_fast,
                                 beta_slow, freq.data_ptr(), ctypes.byref(mscale)),
           "tgdn_rope_freqs")
    return freq.to(device), mscale.value


def rope(q, k, q_out, k_out, freq, *, cu, base=None, off=None, interleaved: bool = False,
         mscale: float = 1.0, transpose: bool = False, stream=None) -> None:
    """tgdn_rope: rotary positions of q [T][H_q][d] and k [T][H_kv][d] (k, k_out may be None)
    into q_out, k_out (the inputs themselves for in place).  The first 2 * len(freq) elements
    of each head are rotated.  Row t of sequence b (cu [B + 1] int32) is at position
    base[b] + off[t] (int32; default: its index within the sequence).  transpose=True is the
    gradient."""
    _check(_native().rope(q, k, q_out, k_out, freq, cu, base, off, interleaved, mscale, transpose,
                          stream), "tgdn_rope")


def prompt_attention_workspace_bytes(B: int, T: int, H_q: int, H_kv: int, d: int) -> int:
    return int(lib().tgdn_prompt_attention_workspace_bytes(B, T, H_q, H_kv, d))


def prompt_attention(cu, q, k, v, o, scale: float, status, ws=None, stream=None) -> None:
    """tgdn_prompt_attention: causal attention over whole prompts packed one after another
    (cu [B + 1] int32).  q, o [T][H_q][d], k, v [T][H_kv][d] (bf16 or f16; rows may be views of
    a fused projection); status [B] int32 is written."""
    _check(_native().prompt_attention(cu, q, k, v, o, scale, status, ws, stream),
           "tgdn_prompt_attention")


class Pages(_Handle):
    """A paged key/value cache's bookkeeping on the device (empty at first), shared by the
    layers: table [B][max_pages], len, held, status [B], refs [n_pages] (int32)."""

    _tensors = ("table", "len", "held", "refs", "status")

    def __init__(self, B: int, n_pages: int, page_size: int, max_pages: int, device="cuda"):
        self.B, self.n_pages = int(B), int(n_pages)
        self.page_size, self.max_pages = int(page_size), int(max_pages)
        new = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        self.table = new(self.B, self.max_pages)
        self.len, self.held, self.status = new(self.B), new(self.B), new(self.B)
        self.refs = new(self.n_pages)

    def _make(self) -> CPages:
        i32, B = torch.int32, self.B
        return CPages(B, self.n_pages, self.page_size, self.max_pages,
                      _dev(self.table, i32, B * self.max_pages, "table"),
                      _dev(self.len, i32, B, "len"), _dev(self.held, i32, B, "held"),
                      _dev(self.refs, i32, self.n_pages, "refs"),
                      _dev(self.status, i32, B, "status"))

    def pool(self, layers: int, H_kv: int, d: int, dtype=torch.bfloat16) -> torch.Tensor:
        """An uninitialised pool [layers][2 (keys, values)][n_pages][H_kv][page_size][d]."""
        return torch.empty((layers, 2, self.n_pages, H_kv, self.page_size, d), dtype=dtype,
                           device=self.table.device)


def _pool(pages: Pages, pool: torch.Tensor) -> torch.Tensor:
    """The pool, if it is one of these pages' kind (its device and layout are checked in C++)."""
    if not isinstance(pool, torch.Tensor) or pool.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("pool: expected a bfloat16 or float16 tensor")
    s = pool.shape
    if len(s) != 6 or s[1] != 2 or s[2] != pages.n_pages or s[4] != pages.page_size:
        raise ValueError(f"pool: shape {tuple(s)}, expected (layers, 2, n_pages, H_kv, page_size, d)")
    return pool


def pages_workspace_bytes(pages: Pages) -> int:
    return int(lib().tgdn_pages_workspace_bytes(ctypes.byref(pages.c())))


def pages_workspace(pages: Pages) -> torch.Tensor:
    """A workspace for the page calls of this cache."""
    n = pages_workspace_bytes(pages)
    if n == 0:
        raise TgdnError(EINVAL, "tgdn_pages_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=pages.table.device)


def pages_reserve(pages: Pages, add, ws, stream=None) -> None:
    """tgdn_pages_reserve: pages for add[b] more positions of every sequence (int32 [B])."""
    _check(_native().pages_reserve(pages, add, ws, stream), "tgdn_pages_reserve")


def pages_append(pages: Pages, cu, k, v, pool, path=None, n_path=None, advance: bool = True,
                 stream=None) -> None:
    """tgdn_pages_append: keys and values k, v [layers][T][H_kv][d] (or [T][H_kv][d] for a pool of
    one layer) to positions len[b], ...: the rows cu[b] .. cu[b+1] - 1, or with path
    [B][path_len] the rows cu[b] + path[b][i], i < n_path[b].  advance=False keeps len."""
    _check(_native().pages_append(pages, cu, k, v, _pool(pages, pool), path, n_path, advance,
                                  stream),
           "tgdn_pages_append")


def pages_fork(pages: Pages, src, dst, pool, status, ws, stream=None) -> None:
    """tgdn_pages_fork: sequence dst[i] becomes a copy of src[i] (int32 [n]); status [n] int32."""
    _check(_native().pages_fork(pages, src, dst, _pool(pages, pool), status, ws, stream),
           "tgdn_pages_fork")


def pages_free(pages: Pages, seq, stream=None) -> None:
    """tgdn_pages_free: releases the pages of the listed sequences (int32)."""
    _check(_native().pages_free(pages, seq, stream), "tgdn_pages_free")


def pages_compact(pages: Pages, pool, n_live, ws, stream=None) -> None:
    """tgdn_pages_compact: live pages to the front of the pool; n_live [1] int32 is written."""
    _check(_native().pages_compact(pages, _pool(pages, pool), n_live, ws, stream),
           "tgdn_pages_compact")


def paged_tree_attention_workspace_bytes(tree: Tree, pages: Pages, H_q: int, H_kv: int,
                                         d: int) -> int:
    return int(lib().tgdn_paged_tree_attention_workspace_bytes(ctypes.byref(tree.c()), H_q, H_kv, d))


def paged_tree_attention(tree: Tree, pages: Pages, q, k_tree, v_tree, k_pages, v_pages, o,
                         scale: float, ws=None, stream=None) -> None:
    """tgdn_paged_tree_attention: each node attends to its sequence's cached positions and its
    own root path.  q/o [T][H_q][d], k_tree/v_tree [T][H_kv][d] (rows may be views of a fused
    projection), k_pages/v_pages [n_pages][H_kv][page_size][d] (one layer of the pool), bf16 or
    f16.  ws: optional workspace of paged_tree_attention_workspace_bytes() bytes, with which
    long contexts are split over CTAs."""
    _check(_native().paged_tree_attention(tree, pages, q, k_tree, v_tree, k_pages, v_pages, o,
                                          scale, ws, stream), "tgdn_paged_tree_attention")


def debug_set_wait_hooks(wait_limit_ns: int = 0, withhold_item: int = -1) -> None:
    """tgdn_debug_set_wait_hooks: a test hook that shortens the bounded device waits of the
    64-node verification kernel and makes its producer withhold one work item's first
    product, so that the consumer's wait expires (TGDN_SEQ_TIMEOUT, no fault or hang).  In
    prompt and paged attention the queries of sequence withhold_item // H_kv, key/value head
    withhold_item % H_kv never come.  debug_set_wait_hooks() restores the defaults."""
    _check(lib().tgdn_debug_set_wait_hooks(int(wait_limit_ns), int(withhold_item)),
           "tgdn_debug_set_wait_hooks")
