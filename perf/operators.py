"""Workloads of the attention-layer operators: rotary positions, attention over packed prompts,
the paged key/value cache, and tree attention over that cache.

Each case is one call (for the cache: one branch's life, or one compaction) as a serving
program makes it.  `own = False` computes it in elementary torch operations, `own = True`
through the library.  `exact` restates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one short chat turn: latency counts
        dict(name="prompt_short", op="prompt", B=1, longest=97, ragged=1, H_q=16, H_kv=4, d=128,
             io="bf16", fused=False),
        # a prefill batch of unequal prompts, q, k, v as views of one fused projection
        dict(name="prompt_ragged", op="prompt", B=16, longest=4001, ragged=2, H_q=16, H_kv=4,
             d=128, io="bf16", fused=True),
        # half-precision layer with one key/value head per query head and small heads
        dict(name="prompt_d64", op="prompt", B=6, longest=2500, ragged=3, H_q=16, H_kv=16, d=64,
             io="fp16", fused=False),
        # one long document
        dict(name="prompt_long", op="prompt", B=1, longest=32768, ragged=4, H_q=16, H_kv=4, d=128,
             io="bf16", fused=False),
        # plain decoding: one new token for one sequence
        dict(name="token_step", op="tree", B=1, longest=1000, ragged=5, N=1, N2=1, H_q=16, H_kv=4,
             d=128, io="bf16", page=64),
        # a verification step: 64-node trees over contexts of up to 4096 positions
        dict(name="tree_step", op="tree", B=16, longest=4096, ragged=6, N=64, N2=64, H_q=16,
             H_kv=4, d=128, io="bf16", page=64),
        # a large mixed batch: 17-node chains and 129-node trees, small pages
        dict(name="tree_mixed", op="tree", B=64, longest=8100, ragged=7, N=129, N2=17, H_q=16,
             H_kv=4, d=128, io="bf16", page=16),
        # single tokens over long contexts
        dict(name="tokens_long", op="tree", B=8, longest=131072, ragged=8, N=1, N2=1, H_q=16,
             H_kv=2, d=128, io="fp16", page=128),
        # a verification step's rotation: tree nodes at cached length + depth
        dict(name="rope_step", op="rope", T=33, B=1, H_q=16, H_kv=4, d=128, rot=128, inter=False,
             scaling="none", factor=1.0, base=5000, io="bf16", fused=False),
        # a long prompt's rotation out of the fused projection, half of each head, long-context scaling
        dict(name="rope_prompt", op="rope", T=16384, B=3, H_q=16, H_kv=4, d=128, rot=64,
             inter=True, scaling="yarn", factor=8.0, base=200000, io="bf16", fused=True),
        # branches of live sequences: forked, extended by an accepted path, dropped
        dict(name="branch", op="branch", B=64, forks=24, L=9, longest=2000, ragged=9, grow=13,
             H_kv=4, d=128, io="bf16", page=64),
        # a fragmented pool moved together
        dict(name="compact", op="compact", B=48, L=9, longest=1500, ragged=10, spare=1.6, H_kv=4,
             d=128, io="bf16", page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "tree", "rope", "rope", "branch", "compact"])
    H_kv = rng.choice([1, 2, 4, 8])
    heads = dict(H_q=H_kv * rng.choice([1, 2, 3, 4, 8]), H_kv=H_kv)
    heads["H_q"] = min(heads["H_q"], 32) // H_kv * H_kv
    ragged = rng.randrange(1 << 30)
    d = rng.choice([64, 128, 128, 96])
    if op == "prompt":
        B = _log(rng, 1, 32)
        longest = _log(rng, 1, 16384 // math.ceil(math.sqrt(B)))
        return dict(op=op, B=B, longest=longest, ragged=ragged, d=d, io=rng.choice(["bf16", "fp16"]),
                    fused=rng.random() < 0.5, **heads)
    if op == "tree":
        B = _log(rng, 1, 64)
        N = rng.choice([1, 1, 7, 33, 64, 129, 200])
        return dict(op=op, B=B, longest=_log(rng, 1, min(65536, 400000 // B)), ragged=ragged, N=N,
                    N2=rng.randint(1, N), d=d, io=rng.choice(["bf16", "fp16"]),
                    page=rng.choice([16, 32, 64, 128, 256]), **heads)
    if op == "rope":
        T = _log(rng, 1, 16384)
        return dict(op=op, T=T, B=min(T, _log(rng, 1, 64)), d=d, rot=rng.choice([d, d, d // 2, 32]),
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), base=_log(rng, 1, 1000000),
                    io=rng.choice(["bf16", "fp16", "fp32"]), fused=rng.random() < 0.5, **heads)
    L = _log(rng, 1, 12)
    B = _log(rng, 2, 64)
    rest = dict(L=L, B=B, longest=_log(rng, 1, 2000), ragged=ragged, H_kv=H_kv, d=d,
                io=rng.choice(["bf16", "fp16"]), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "branch":
        return dict(op=op, forks=rng.randint(1, B // 2), grow=rng.randint(1, 31), **rest)
    return dict(op=op, spare=rng.choice([1.1, 1.5, 2.5]), **rest)


# ---------------------------------------------------------------------------- shapes
def _lengths(c, n=None):
    """The longest, then lengths spread over their logarithm (one-token and empty ones too)."""
    r = random.Random(c["ragged"])
    out = [c["longest"]]
    for i in range(1, n or c["B"]):
        out.append(0 if i % 13 == 12 else int(round(math.exp(r.uniform(0, math.log(c["longest"]))))))
    if c["op"] == "prompt":  # every other prompt is of the longest one's order
        out = [max(x, c["longest"] // 3) if i % 2 == 1 else x for i, x in enumerate(out)]
    else:  # most contexts are of one order
        out = [max(x, c["longest"] // 2) if i % 4 != 3 else x for i, x in enumerate(out)]
    return out


def _trees(c):
    """Parents of each sequence's tree: N and N2 nodes in turn, each under a random earlier one."""
    r = random.Random(c["ragged"] + 1)
    trees = []
    for b in range(c["B"]):
        parent, depth = [-1], [0]
        for i in range(1, c["N"] if b % 2 == 0 else c["N2"]):
            p = r.randrange(max(0, i - 8), i)
            while depth[p] >= 30:
                p = parent[p]
            parent.append(p)
            depth.append(depth[p] + 1)
        trees.append((parent, depth))
    return trees


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _rope_rows(c):
    """Rows of each sequence and the position of its first row."""
    T, B = c["T"], c["B"]
    cu = [T * b // B for b in range(B + 1)]
    return cu, [c["base"] // (b + 1) for b in range(B)]


def _rand(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _inv_freq(c):
    """Radians per position of each pair, and the factor on the rotated values."""
    rot, theta, s = c["rot"], 10000.0, c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if c["scaling"] == "ntk":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "yarn":  # fast pairs kept, slow ones interpolated, a ramp between
        def pair(turns):
            return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    return f, 1.0


# ---------------------------------------------------------------------------- inputs
def _prompt_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = _lengths(c)
    T, H_q, H_kv, d, dt = sum(lens), c["H_q"], c["H_kv"], c["d"], DTYPES[c["io"]]
    if c["fused"]:
        qkv = _rand(g, (T, H_q + 2 * H_kv, d), dt)
        qkv[:, :H_q] *= 2
        q, k, v = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
    else:
        q, k, v = _rand(g, (T, H_q, d), dt, 2.0), _rand(g, (T, H_kv, d), dt), _rand(g, (T, H_kv, d), dt)
    return dict(c=c, lens=lens, cu=_ints(_cu(lens)), q=q, k=k, v=v, scale=d ** -0.5)


def _tree_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, trees, ps, dt = _lengths(c), _trees(c), c["page"], DTYPES[c["io"]]
    B, H_q, H_kv, d = c["B"], c["H_q"], c["H_kv"], c["d"]
    held = [-(-n // ps) for n in lens]
    n_pages = sum(held) + 5
    cu = _cu([len(p) for p, _ in trees])
    T, nmax = cu[-1], max(c["N"], c["N2"])
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(max(held), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    sees = torch.zeros((B, nmax, nmax), dtype=torch.bool)
    for b, (parent, _) in enumerate(trees):
        for n, p in enumerate(parent):
            if p >= 0:
                sees[b, n] = sees[b, p]
            sees[b, n, n] = True
    pool = _rand(g, (2, n_pages, H_kv, ps, d), dt)
    return dict(c=c, lens=lens, held=held, cu_list=cu, trees=trees, nmax=nmax, table=table,
                sees=sees.cuda(), k_pages=pool[0], v_pages=pool[1], n_pages=n_pages,
                q=_rand(g, (T, H_q, d), dt, 2.0), k=_rand(g, (T, H_kv, d), dt),
                v=_rand(g, (T, H_kv, d), dt), scale=d ** -0.5)


def _rope_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu, base = _rope_rows(c)
    T, H_q, H_kv, d, dt = c["T"], c["H_q"], c["H_kv"], c["d"], DTYPES[c["io"]]
    if c["fused"]:
        qkv = _rand(g, (T, H_q + 2 * H_kv, d), dt)
        q, k = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv]
    else:
        q, k = _rand(g, (T, H_q, d), dt), _rand(g, (T, H_kv, d), dt)
    r = random.Random(seed)  # tree nodes: each at the depth of some walk from its root
    off = []
    for b in range(c["B"]):
        n = cu[b + 1] - cu[b]
        off += list(range(n)) if n > 256 else [r.randint(0, min(i, 30)) for i in range(n)]
    return dict(c=c, q=q, k=k, cu=_ints(cu), base=_ints(base), off=_ints(off))


def _pool_inputs(c, seed):
    """A pool whose live sequences hold scattered pages."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(c["ragged"] + 2)
    ps, B, dt = c["page"], c["B"], DTYPES[c["io"]]
    lens = _lengths(c)
    live = B // 2 if c["op"] == "branch" else B
    lens = [max(n, 1) if b < live else 0 for b, n in enumerate(lens)]
    held = [-(-n // ps) for n in lens]
    grow = c.get("grow", 0)
    max_pages = max(held) + -(-grow // ps) + 1
    extra = c.get("forks", 0) * (2 + -(-grow // ps))
    n_pages = int(sum(held) * c.get("spare", 1.3)) + extra + 3
    ids = r.sample(range(n_pages), sum(held))
    table, at = [], 0
    refs = [0] * n_pages
    for b in range(B):
        row = ids[at:at + held[b]]
        at += held[b]
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (max_pages - held[b]))
    pool = _rand(g, (c["L"], 2, n_pages, c["H_kv"], ps, c["d"]), dt)
    s = dict(c=c, pool=pool, table=_ints(table), len=_ints(lens), held=_ints(held), refs=_ints(refs),
             n_pages=n_pages, max_pages=max_pages)
    if c["op"] == "branch":
        n = c["forks"]
        src = [r.randrange(live) for _ in range(n)]
        dst = r.sample(range(live, B), n)
        depth, count = 31, [0] * B
        for b in dst:
            count[b] = r.randint(1, grow)
        rows = [2 * x for x in count]  # a tree of twice the accepted path's nodes
        cu = _cu(rows)
        path = [sorted(r.sample(range(rows[b]), count[b])) + [-1] * (depth - count[b]) for b in range(B)]
        T = max(cu[-1], 1)
        s.update(src=_ints(src), dst=_ints(dst), add=_ints(count), cu=_ints(cu), path=_ints(path),
                 k=_rand(g, (c["L"], T, c["H_kv"], c["d"]), dt),
                 v=_rand(g, (c["L"], T, c["H_kv"], c["d"]), dt), T=T)
    else:
        s.update(table0=s["table"].clone(), refs0=s["refs"].clone())
    return s


def prepare(case, seed):
    make = {"prompt": _prompt_inputs, "tree": _tree_inputs, "rope": _rope_inputs,
            "branch": _pool_inputs, "compact": _pool_inputs}[case["op"]]
    s = make(case, seed)
    if case["op"] == "rope":
        s["inv_freq"], s["mscale"] = _inv_freq(case)
        s["inv_freq"] = s["inv_freq"].cuda()
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    from tree_speculative_decoding_gated_gb300 import tgdn
    c = s["c"]
    s["tgdn"] = tgdn
    if c["op"] in ("prompt", "tree"):
        s["o"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    if c["op"] == "prompt":
        s["status"] = torch.empty(c["B"], dtype=torch.int32, device="cuda")
        n = tgdn.prompt_attention_workspace_bytes(c["B"], s["q"].shape[0], c["H_q"], c["H_kv"], c["d"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    elif c["op"] == "tree":
        parents = [p for tree, _ in s["trees"] for p in tree]
        s["tree"] = tgdn.Tree.from_host(s["cu_list"], parents, s["nmax"], 30)
        tgdn.tree_prep(s["tree"])
        s["pages"] = tgdn.Pages(c["B"], s["n_pages"], c["page"], s["table"].shape[1])
        s["pages"].table.copy_(s["table"])
        s["pages"].len.copy_(_ints(s["lens"]))
        s["pages"].held.copy_(_ints(s["held"]))
        n = tgdn.paged_tree_attention_workspace_bytes(s["tree"], s["pages"], c["H_q"], c["H_kv"], c["d"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    elif c["op"] == "rope":
        s["freq"], s["mscale"] = tgdn.rope_freqs(c["rot"], 10000.0, c["scaling"], c["factor"], 4096)
        s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        s["k_out"] = torch.empty(s["k"].shape, dtype=s["k"].dtype, device="cuda")
    else:
        p = s["pages"] = tgdn.Pages(c["B"], s["n_pages"], c["page"], s["max_pages"])
        for name in ("table", "len", "held", "refs"):
            getattr(p, name).copy_(s[name])
        s["ws"] = tgdn.pages_workspace(p)
        s["fork_status"] = torch.zeros(c.get("forks", 1), dtype=torch.int32, device="cuda")
        s["n_live"] = torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)[s["c"]["op"]](s)


def _prompt_own(s):
    s["tgdn"].prompt_attention(s["cu"], s["q"], s["k"], s["v"], s["o"], s["scale"], s["status"], ws=s["ws"])
    return s["o"]


def _tree_own(s):
    s["tgdn"].paged_tree_attention(s["tree"], s["pages"], s["q"], s["k"], s["v"], s["k_pages"],
                                   s["v_pages"], s["o"], s["scale"], ws=s["ws"])
    return s["o"]


def _rope_own(s):
    s["tgdn"].rope(s["q"], s["k"], s["q_out"], s["k_out"], s["freq"], interleaved=s["c"]["inter"],
                   mscale=s["mscale"], cu=s["cu"], base=s["base"], off=s["off"])
    return [s["q_out"], s["k_out"]]


def _branch_own(s):
    t, p = s["tgdn"], s["pages"]
    t.pages_fork(p, s["src"], s["dst"], s["pool"], s["fork_status"], s["ws"])
    t.pages_reserve(p, s["add"], s["ws"])
    t.pages_append(p, s["cu"], s["k"], s["v"], s["pool"], path=s["path"], n_path=s["add"])
    t.pages_free(p, s["dst"])
    return [s["pool"], p.table, p.len, p.held, p.refs, s["fork_status"]]


def _compact_own(s):
    t, p = s["tgdn"], s["pages"]
    p.table.copy_(s["table0"])
    p.refs.copy_(s["refs0"])
    t.pages_compact(p, s["pool"], s["n_live"], s["ws"])
    return [s["pool"], p.table, p.refs, s["n_live"]]


def _softmax_av(x, seen, v):
    """softmax over the seen keys (zero where none is) times v, in 32 bits."""
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, torch.ones_like(total), total)


def _prompt_plain(s):
    c, at = s["c"], 0
    H_q, H_kv, d = c["H_q"], c["H_kv"], c["d"]
    G, out = H_q // H_kv, torch.zeros(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    for n in s["lens"]:
        for h in range(H_kv if n else 0):
            k, v = (s[x][at:at + n, h].float() for x in "kv")
            for i in range(0, n, 2048):
                j = min(n, i + 2048)
                q = s["q"][at + i:at + j, h * G:(h + 1) * G].float().reshape(-1, d)
                row = torch.arange(i, j, device="cuda").repeat_interleave(G)
                seen = torch.arange(j, device="cuda")[None, :] <= row[:, None]
                o = _softmax_av(q @ k[:j].T * s["scale"], seen, v[:j])
                out[at + i:at + j, h * G:(h + 1) * G] = o.reshape(j - i, G, d).to(out.dtype)
        at += n
    return out


def _tree_plain(s):
    c, cu = s["c"], s["cu_list"]
    H_q, H_kv, d, ps = c["H_q"], c["H_kv"], c["d"], c["page"]
    G, out = H_q // H_kv, torch.zeros(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    for b in range(c["B"]):
        lo, hi, P = cu[b], cu[b + 1], s["lens"][b]
        N, ids = hi - lo, s["table"][b, :s["held"][b]].long()
        seen = torch.cat([torch.ones((N, P), dtype=torch.bool, device="cuda"), s["sees"][b, :N, :N]], 1)
        seen = seen.repeat_interleave(G, 0)
        for h in range(H_kv):
            k, v = (torch.cat([s[x + "_pages"][ids, h].reshape(-1, d)[:P], s[x][lo:hi, h]]).float()
                    for x in "kv")
            q = s["q"][lo:hi, h * G:(h + 1) * G].float().reshape(-1, d)
            o = _softmax_av(q @ k.T * s["scale"], seen, v)
            out[lo:hi, h * G:(h + 1) * G] = o.reshape(N, G, d).to(out.dtype)
    return out


def _rope_plain(s):
    c = s["c"]
    rot = c["rot"]
    n = s["cu"][1:] - s["cu"][:-1]
    pos = torch.repeat_interleave(s["base"], n, output_size=c["T"]) + s["off"]
    angle = pos.double()[:, None] * s["inv_freq"][None, :]
    cos, sin = ((f(angle) * s["mscale"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    outs = []
    for x in (s["q"], s["k"]):
        y = x.float().clone()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        u, w = a * cos - b * sin, a * sin + b * cos
        a.copy_(u)
        b.copy_(w)
        outs.append(y.to(x.dtype))
    return outs


def _free_pages(refs, n):
    """The n lowest free pages."""
    return torch.argsort((refs != 0).to(torch.int8), stable=True)[:n]


def _branch_plain(s):
    c = s["c"]
    ps, pool, table, ln, held, refs = c["page"], s["pool"], s["table"], s["len"], s["held"], s["refs"]
    src, dst, cols = s["src"].long(), s["dst"].long(), torch.arange(s["max_pages"], device="cuda")
    # fork: whole pages shared, the last, partly filled one copied
    full, tail = ln[src] // ps, ln[src] % ps
    has = tail > 0
    free = _free_pages(refs, int(src.numel()))
    new = free[(torch.cumsum(has, 0) - 1).clamp(min=0)].int()
    old = table[src, full.long().clamp(max=s["max_pages"] - 1)]
    rows = torch.where(cols[None] < full[:, None], table[src], table[dst])
    last = (cols[None] == full[:, None]) & has[:, None]
    table[dst] = torch.where(last, new[:, None], rows)
    share = cols[None] < full[:, None]
    refs.index_add_(0, table[src].clamp(min=0).reshape(-1).long(), share.reshape(-1).int())
    refs.index_add_(0, new.long(), has.int())
    ln[dst] = ln[src]
    held[dst] = full + has.int()
    pick = has.nonzero()[:, 0]
    keep = torch.arange(ps, device="cuda")[None] < tail[pick][:, None]
    a, b = old[pick].long(), new[pick].long()
    pool[:, :, b] = torch.where(keep[:, None, :, None], pool[:, :, a], pool[:, :, b])
    # reserve room for the accepted paths
    need = (ln + s["add"] + ps - 1) // ps
    more = (need - held).clamp(min=0)
    take = (cols[None] >= held[:, None]) & (cols[None] < (held + more)[:, None])
    where = take.nonzero()
    free = _free_pages(refs, where.shape[0])
    table[where[:, 0], where[:, 1]] = free.int()
    refs[free] = 1
    held += more
    # append them
    item = torch.arange(s["path"].shape[1], device="cuda")
    b, i = (item[None] < s["add"][:, None]).nonzero().T
    row = (s["cu"][b] + s["path"][b, i]).long()
    at = ln[b] + i
    page = table[b, (at // ps).long()].long()
    pool[:, 0, page, :, (at % ps).long()] = s["k"][:, row].transpose(0, 1)
    pool[:, 1, page, :, (at % ps).long()] = s["v"][:, row].transpose(0, 1)
    ln += s["add"]
    # and free the branches
    mine = cols[None] < held[dst][:, None]
    refs.index_add_(0, table[dst].clamp(min=0).reshape(-1).long(), -mine.reshape(-1).int())
    ln[dst] = 0
    held[dst] = 0
    return [pool, table, ln, held, refs, torch.zeros(src.numel(), dtype=torch.int32, device="cuda")]


def _compact_plain(s):
    pool, table, refs = s["pool"], s["table"], s["refs"]
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    idx = torch.arange(s["n_pages"], device="cuda")
    n_live = (refs > 0).sum()
    movers = ((refs > 0) & (idx >= n_live)).nonzero()[:, 0]
    holes = ((refs == 0) & (idx < n_live)).nonzero()[:, 0]
    to = idx.clone()
    to[movers] = holes
    mine = torch.arange(s["max_pages"], device="cuda")[None] < s["held"][:, None]
    table.copy_(torch.where(mine, to[table.clamp(min=0).long()].int(), table))
    refs[holes] = refs[movers]
    refs[movers] = 0
    pool[:, :, holes] = pool[:, :, movers]
    return [pool, table, refs, n_live.int().reshape(1)]


_plain = dict(prompt=_prompt_plain, tree=_tree_plain, rope=_rope_plain, branch=_branch_plain, compact=_compact_plain)
_own = dict(prompt=_prompt_own, tree=_tree_own, rope=_rope_own, branch=_branch_own, compact=_compact_own)


# ---------------------------------------------------------------------------- least work
def work(case):
    c = case
    es = 4 if c["io"] == "fp32" else 2
    if c["op"] == "prompt":
        lens = _lengths(c)
        rows = sum(lens) * c["d"] * es
        return dict(bytes=rows * 2 * (c["H_q"] + c["H_kv"]),
                    flops=4 * c["d"] * c["H_q"] * sum(n * (n + 1) // 2 for n in lens))
    if c["op"] == "tree":
        lens, trees = _lengths(c), _trees(c)
        T = sum(len(p) for p, _ in trees)
        keys = sum(len(p) * n + sum(x + 1 for x in dep) for n, (p, dep) in zip(lens, trees))
        return dict(bytes=c["d"] * es * (2 * c["H_kv"] * sum(lens) + 2 * T * (c["H_q"] + c["H_kv"]))
                    + 4 * sum(-(-n // c["page"]) for n in lens), flops=4 * c["d"] * c["H_q"] * keys)
    heads = c.get("H_q", 0) + c["H_kv"]
    if c["op"] == "rope":
        return dict(bytes=2 * c["T"] * heads * c["d"] * es + 4 * c["T"],
                    flops=3 * c["T"] * heads * c["rot"])
    lens, ps = _lengths(c), c["page"]
    pos = 2 * c["L"] * c["H_kv"] * c["d"] * es  # a position's keys and values in every layer
    r = random.Random(c["ragged"] + 2)
    live = c["B"] // 2 if c["op"] == "branch" else c["B"]
    lens = [max(n, 1) if b < live else 0 for b, n in enumerate(lens)]
    held = sum(-(-n // ps) for n in lens)
    extra = c.get("forks", 0) * (2 + -(-c.get("grow", 0) // ps))
    n_pages = int(held * c.get("spare", 1.3)) + extra + 3
    ids = r.sample(range(n_pages), held)
    if c["op"] == "compact":
        moved = sum(1 for p in ids if p >= held)
        return dict(bytes=2 * moved * ps * pos + 8 * (n_pages + held), flops=0)
    src = [r.randrange(live) for _ in range(c["forks"])]
    r.sample(range(live, c["B"]), c["forks"])
    new = sum(r.randint(1, c["grow"]) for _ in range(c["forks"]))
    return dict(bytes=2 * pos * (sum(lens[b] % ps for b in src) + new)
                + 8 * sum(-(-lens[b] // ps) for b in src) + 4 * n_pages, flops=0)


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = case
    if c["op"] in ("branch", "compact"):
        return None  # copies and whole numbers
    if c["op"] == "rope":
        return _rope_exact(c, seed)
    return _prompt_exact(c, seed) if c["op"] == "prompt" else _tree_exact(c, seed)


def _attend(q, k, v, hidden, scale):
    """q [h][n][d], k and v [keys][d], hidden [n][keys]: in 64 bits."""
    w = torch.einsum("hnd,kd->hnk", q.double(), k.double()).mul_(scale)
    w.masked_fill_(hidden[None], -math.inf)
    return torch.einsum("hnk,kd->hnd", torch.softmax(w, dim=2), v.double())


def _prompt_exact(c, seed):
    s = _prompt_inputs(c, seed)
    per, cu = c["H_q"] // c["H_kv"], _cu(s["lens"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for lo, hi in zip(cu[:-1], cu[1:]):
        for first in range(lo, hi, 1024):
            last = min(first + 1024, hi)
            hidden = torch.ones((last - first, last - lo), dtype=torch.bool, device="cuda").triu(first - lo + 1)
            for h in range(c["H_kv"]):
                hs = slice(h * per, h * per + per)
                y = _attend(s["q"][first:last, hs].permute(1, 0, 2), s["k"][lo:last, h], s["v"][lo:last, h],
                            hidden, s["scale"])
                out[first:last, hs] = y.permute(1, 0, 2)
    return out


def _tree_exact(c, seed):
    s = _tree_inputs(c, seed)
    per, ps = c["H_q"] // c["H_kv"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (parent, _) in enumerate(s["trees"]):
        lo, hi, P = s["cu_list"][b], s["cu_list"][b + 1], s["lens"][b]
        hidden = torch.zeros((hi - lo, P + hi - lo), dtype=torch.bool)
        hidden[:, P:] = True
        for n in range(hi - lo):
            a = n
            while a >= 0:
                hidden[n, P + a] = False
                a = parent[a]
        at = torch.arange(P, device="cuda")
        page, inside = s["table"][b][at // ps].long(), at % ps
        for h in range(c["H_kv"]):
            hs = slice(h * per, h * per + per)
            k = torch.cat([s["k_pages"][page, h, inside], s["k"][lo:hi, h]])
            v = torch.cat([s["v_pages"][page, h, inside], s["v"][lo:hi, h]])
            y = _attend(s["q"][lo:hi, hs].permute(1, 0, 2), k, v, hidden.cuda(), s["scale"])
            out[lo:hi, hs] = y.permute(1, 0, 2)
    return out


def _rope_exact(c, seed):
    s = _rope_inputs(c, seed)
    f, m = _inv_freq(c)
    cu, base = _rope_rows(c)
    start = torch.cat([torch.full((cu[b + 1] - cu[b],), base[b]) for b in range(c["B"])]).cuda()
    turn = torch.polar(torch.full((), m, dtype=torch.float64, device="cuda"),
                       torch.outer((start + s["off"]).double(), f.cuda()))[:, None]
    outs, half = [], c["rot"] // 2
    for x in (s["q"], s["k"]):
        y = x.double()
        z = y[..., :c["rot"]]
        if c["inter"]:
            z = torch.view_as_real(torch.view_as_complex(z.reshape(*z.shape[:2], half, 2).contiguous()) * turn)
            z = z.reshape(*y.shape[:2], -1)
        else:
            z = torch.complex(z[..., :half], z[..., half:]) * turn
            z = torch.cat([z.real, z.imag], -1)
        outs.append(torch.cat([z, y[..., c["rot"]:]], -1))
    return outs
