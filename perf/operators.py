"""Cases of the paged-cache operators: what each is timed on, and its plain form.

Five operators over a KV cache held in pages (slot s of request b is row
``s % page_size`` of page ``block_table[b, s // page_size]``):

    attention  tree_attention_paged: the tree tokens over prefix + tree
    rope       qk_rope_append: per-head norms, rotation, K/V into the pages
    commit     tree_commit_paged: the accepted path's K/V next to the prefix
    resize     pages_resize: pages for the coming step, then back
    fork       pages_fork: a sequence continued twice, its last page copied

``run`` computes them with elementary torch operations (``own`` false) or with
the package's kernels (``own`` true) on what ``prepare`` made.
"""
import math

import torch

own = False

DEV = "cuda"
KPH = (10, 10, 10, 10)          # candidates of each draft head, as the package's workloads have them


# ------------------------------------------------------------------ the cases

def listed():
    att = dict(op="attention", tree="topk", out="bf16")
    return [
        # the smallest verification step of the package's tiny workload: latency
        dict(att, name="attention-tiny", B=1, T=17, Hq=4, Hkv=2, dh=64, page=16, lo=128, hi=128, out="fp32"),
        # one 70B-shaped request with its 64-candidate tree
        dict(att, name="attention-70b-tree", B=1, T=65, Hq=64, Hkv=8, dh=128, page=64, lo=4096, hi=4096),
        # a batch of them with ragged prefixes: the tensor cores' case
        dict(att, name="attention-70b-b8", B=8, T=65, Hq=64, Hkv=8, dh=128, page=64, lo=1024, hi=8192),
        # plain decoding (a tree of one node) of 8B-shaped requests over long contexts: the memory's case
        dict(att, name="attention-decode-long", B=16, T=1, Hq=32, Hkv=8, dh=128, page=16, lo=20001, hi=32768),
        # the tree's queries and keys of one step, norms and rotation, into the pages
        dict(name="rope-tree", op="rope", B=1, T=65, Hq=64, Hkv=8, dh=128, page=64, lo=4096, hi=4096, rot=128,
             norm=True, pairs="half", ragged=False),
        # padded prompts of several requests at the start of their sequences
        dict(name="rope-prompt", op="rope", B=8, T=4096, Hq=32, Hkv=8, dh=128, page=16, lo=0, hi=0, rot=128,
             norm=True, pairs="half", ragged=True),
        # the accepted path of one request in every layer
        dict(name="commit-b1", op="commit", B=1, T=65, L=80, Hkv=8, dh=128, page=64, lo=500, hi=500),
        # the same for a batch
        dict(name="commit-b32", op="commit", B=32, T=65, L=32, Hkv=8, dh=128, page=16, lo=40, hi=400),
        # a step's pages reserved and given back, small server
        dict(name="resize-b8", op="resize", B=8, T=65, page=16, lo=1024, hi=8192, spare=1.25),
        # the same for a server of many requests and a large pool
        dict(name="resize-b256", op="resize", B=256, T=65, page=16, lo=100, hi=16384, spare=1.5),
        # one sequence forked into four
        dict(name="fork-b4", op="fork", B=5, n=4, one=True, L=32, Hkv=8, dh=128, page=64, lo=200, hi=500),
        # half of a batch forked into its other half
        dict(name="fork-b32", op="fork", B=32, n=16, one=False, L=32, Hkv=8, dh=128, page=64, lo=70, hi=700),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rope", "commit", "resize", "fork"])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([(4, 2, 64), (8, 8, 64), (32, 8, 128), (64, 8, 128), (28, 4, 128), (16, 1, 64), (12, 4, 64),
                        (40, 8, 128)])
    Hq, Hkv, dh = heads
    while True:
        if op == "attention":
            lo = _log(rng, 1, 32768) - 1
            c = dict(op=op, B=_log(rng, 1, 32), T=rng.choice([1, 2, 5, 17, rng.randint(2, 128), 65]), Hq=Hq, Hkv=Hkv,
                     dh=dh, page=page, lo=lo, hi=rng.randint(lo, 32768 if rng.random() < 0.3 else 2 * lo + 16),
                     tree=rng.choice(["topk", "chain"]), out=rng.choice(["bf16", "bf16", "fp32"]))
            if c["tree"] == "chain":
                c["T"] = min(c["T"], 5)
        elif op == "rope":
            lo = _log(rng, 1, 100000) - 1
            c = dict(op=op, B=_log(rng, 1, 16), T=_log(rng, 1, 4096), Hq=Hq, Hkv=Hkv, dh=dh, page=page, lo=lo,
                     hi=lo + rng.randint(0, 1000), rot=rng.choice([dh, dh, dh // 2]), norm=rng.random() < 0.6,
                     pairs=rng.choice(["half", "half", "adjacent"]), ragged=rng.random() < 0.5)
        elif op == "commit":
            lo = _log(rng, 1, 400)
            c = dict(op=op, B=_log(rng, 1, 32), T=rng.randint(2, 128), L=_log(rng, 1, 80), Hkv=Hkv, dh=dh, page=page,
                     lo=lo, hi=lo + rng.randint(0, 200))
        elif op == "resize":
            lo = _log(rng, 1, 8192)
            c = dict(op=op, B=_log(rng, 1, 256), T=rng.randint(1, 128), page=page, lo=lo, hi=rng.randint(lo, 16384),
                     spare=rng.choice([1.0, 1.25, 1.5]))
        else:
            one = rng.random() < 0.5
            n = _log(rng, 1, 16)
            lo = _log(rng, 1, 500)
            c = dict(op=op, B=n + 1 if one else 2 * n, n=n, one=one, L=_log(rng, 1, 32), Hkv=Hkv, dh=dh, page=page,
                     lo=lo, hi=lo + rng.randint(0, 200))
        caps = [x for x in listed() if x["op"] == op]
        w = work(c)
        fits = all(w[k] <= max(work(x)[k] for x in caps) for k in ("bytes", "flops"))
        if fits and _pool_bytes(c) <= max(_pool_bytes(x) for x in listed()):
            return c


# ------------------------------------------------- what follows from a case alone

def _lengths(c):
    """Prefix lengths of the requests: spread over [lo, hi]."""
    return [c["lo"] + int((c["hi"] - c["lo"]) * ((b * 0.6180339887498949) % 1.0 if c["B"] > 1 else 1.0))
            for b in range(c["B"])]


def _new_tokens(c):
    """Tokens of each request of a padded batch of T columns."""
    return [max(1, c["T"] - (b * 997) % (c["T"] // 2 + 1)) if c["ragged"] else c["T"] for b in range(c["B"])]


def _tree(T, kind):
    """parent and head rank of each node, root first, by depth: a chain, or the
    candidates of four heads in the order of the rank sums (ten a head)."""
    if kind == "chain":
        return [-1] + list(range(T - 1)), [0] * T
    nodes = [()]
    frontier = [(0, ())]
    while len(nodes) < T:
        nxt = min(((sum(t) + 1.5 * len(t) + r + 1.0, t + (r,)) for _, t in frontier if len(t) < len(KPH)
                   for r in [sum(1 for n in nodes if len(n) == len(t) + 1 and n[:-1] == t)] if r < KPH[len(t)]),
                  key=lambda x: (x[0], x[1]))
        nodes.append(nxt[1])
        frontier.append((0, nxt[1]))
    nodes.sort(key=lambda t: (len(t), t))
    index = {t: j for j, t in enumerate(nodes)}
    return [-1] + [index[t[:-1]] for t in nodes[1:]], [0] + [t[-1] for t in nodes[1:]]


def _depths(parent):
    d = [0] * len(parent)
    for j in range(1, len(parent)):
        d[j] = d[parent[j]] + 1
    return d


def _paths(c, parent):
    """An accepted path of each request: any node's whose sources are not also
    slots written for another node, so that a pass may be repeated."""
    good = []
    for j in range(len(parent)):
        p, n = [], j
        while n >= 0:
            p.insert(0, n)
            n = parent[n]
        if all(x == i or x >= len(p) for i, x in enumerate(p)):
            good.append(p)
    return [good[(7 + 13 * b) % len(good)] for b in range(c["B"])]


def _pages(n, page):
    return (n + page - 1) // page


def _pool_pages(c):
    ln = _lengths(c)
    if c["op"] == "rope":
        # only the slots written lie in pages of their own; the prefix shares one
        return sum(_pages(p + n, c["page"]) - p // c["page"] for p, n in zip(ln, _new_tokens(c))) + 1
    if c["op"] == "fork":
        return sum(_pages(p, c["page"]) for p in ln) + c["n"] + 3
    if c["op"] == "resize":
        return int(c["spare"] * sum(_pages(p + c["T"], c["page"]) for p in ln)) + 1
    return sum(_pages(p + c["T"], c["page"]) for p in ln) + 2


def _pool_bytes(c):
    if c["op"] == "resize":
        return 4 * _pool_pages(c)
    return 4 * c.get("L", 1) * _pool_pages(c) * c["Hkv"] * c["page"] * c["dh"]


def work(case):
    c, ln = case, _lengths(case)
    if c["op"] == "attention":
        parent, _ = _tree(c["T"], c["tree"])
        seen = sum(d + 1 for d in _depths(parent))
        pairs = sum(c["T"] * p + seen for p in ln)
        rows = c["B"] * c["T"] * c["Hq"] * c["dh"]
        return {"bytes": 4 * c["Hkv"] * c["dh"] * sum(p + c["T"] for p in ln) + rows * (2 + (4 if c["out"] == "fp32" else 2))
                + 4 * sum(_pages(p + c["T"], c["page"]) for p in ln),
                "flops": 4 * c["Hq"] * c["dh"] * pairs}
    if c["op"] == "rope":
        n = sum(_new_tokens(c))
        return {"bytes": n * (4 * (c["Hq"] + 2 * c["Hkv"]) * c["dh"] + 4),
                "flops": n * (c["Hq"] + c["Hkv"]) * c["dh"] * (8 if c["norm"] else 4)}
    if c["op"] == "commit":
        parent, _ = _tree(c["T"], "topk")
        moved = sum(sum(1 for i, x in enumerate(p) if x != i) for p in _paths(c, parent))
        return {"bytes": 8 * c["L"] * c["Hkv"] * c["dh"] * moved + 40 * c["B"], "flops": 0}
    if c["op"] == "resize":
        new = sum(_pages(p + c["T"], c["page"]) - _pages(p, c["page"]) for p in ln)
        return {"bytes": 2 * (4 * _pool_pages(c) + 12 * c["B"] + 8 * new), "flops": 0}
    src = _fork_rows(c)[0]
    rows = sum(ln[s] % c["page"] for s in src)
    shared = sum(ln[s] // c["page"] for s in src)
    return {"bytes": 8 * c["L"] * c["Hkv"] * c["dh"] * rows + 16 * shared + 4 * _pool_pages(c), "flops": 0}


def _fork_rows(c):
    if c["one"]:
        return [0] * c["n"], [1 + i for i in range(c["n"])]
    return list(range(c["n"])), [c["n"] + i for i in range(c["n"])]


# ------------------------------------------------------------------- inputs

def _normal(g, *shape):
    """N(0, 1) in bf16."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV)
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _scattered_table(g, counts, width, n_pool):
    """Pages in the order a long-running server has them: none in particular."""
    perm = torch.randperm(n_pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _inputs(c, seed):
    """The inputs of a case, from the seed alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ln, page = _lengths(c), c["page"]
    N = _pool_pages(c)
    s = dict(case=c, lens=ln, prefix_len=_i32(ln), N=N)
    if c["op"] == "attention":
        s["parent"], s["rank"] = _tree(c["T"], c["tree"])
        see = torch.eye(c["T"], dtype=torch.bool)
        for t in range(1, c["T"]):
            see[t] |= see[s["parent"][t]]
        s["hide"] = ~see.to(DEV)                 # nodes of the tree that a node does not see
        counts = [_pages(p + c["T"], page) for p in ln]
        s["block_table"] = _scattered_table(g, counts, max(counts), N)
        s["q"] = _normal(g, c["B"], c["T"], c["Hq"], c["dh"])
        s["k_pages"] = _normal(g, N, c["Hkv"], page, c["dh"])
        s["v_pages"] = _normal(g, N, c["Hkv"], page, c["dh"])
    elif c["op"] == "rope":
        new = _new_tokens(c)
        # the fused projection's output; q, k and v are views of it
        qkv = _normal(g, c["B"], c["T"], c["Hq"] + 2 * c["Hkv"], c["dh"])
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
        s["q_norm"] = (1.0 + 0.2 * _normal(g, c["dh"])).bfloat16() if c["norm"] else None
        s["k_norm"] = (1.0 + 0.2 * _normal(g, c["dh"])).bfloat16() if c["norm"] else None
        half = c["rot"] // 2
        s["inv_freq"] = (500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEV)
        offs = torch.arange(c["T"], dtype=torch.int32, device=DEV)
        s["pos"] = s["prefix_len"][:, None] + offs[None, :]
        s["new_list"], s["n_new"] = new, _i32(new) if c["ragged"] else None
        width = max(_pages(p + n, page) for p, n in zip(ln, new))
        perm = (torch.randperm(N - 1, generator=g, device=DEV) + 1).to(torch.int32)
        table = torch.zeros((c["B"], width), dtype=torch.int32, device=DEV)
        at = 0
        for b, (p, n) in enumerate(zip(ln, new)):
            first, last = p // page, _pages(p + n, page)
            table[b, first:last] = perm[at:at + last - first]
            table[b, last:] = -1
            at += last - first
        s["block_table"] = table
        s["k_pages"] = _normal(g, N, c["Hkv"], page, c["dh"])
        s["v_pages"] = _normal(g, N, c["Hkv"], page, c["dh"])
    elif c["op"] == "commit":
        s["parent"], s["rank"] = _tree(c["T"], "topk")
        paths = _paths(c, s["parent"])
        counts = [_pages(p + c["T"], page) for p in ln]
        s["block_table"] = _scattered_table(g, counts, max(counts), N)
        s["accept_len"] = _i32([len(p) - 1 for p in paths])
        s["path"] = _i32([p + [-1] * (len(KPH) + 1 - len(p)) for p in paths])
        s["bonus"] = torch.randint(0, 128256, (c["B"],), generator=g, device=DEV, dtype=torch.int32)
        s["k_pages"] = _normal(g, c["L"], N, c["Hkv"], page, c["dh"])
        s["v_pages"] = _normal(g, c["L"], N, c["Hkv"], page, c["dh"])
    else:
        counts = [_pages(p, page) for p in ln]
        if c["op"] == "fork":
            s["src_list"], s["dst_list"] = _fork_rows(c)
            s["src"], s["dst"] = _i32(s["src_list"]), _i32(s["dst_list"])
            width = max(counts) + 1
            # rows about to be written hold an older sequence, or nothing
            s["k_pages"] = _normal(g, c["L"], N, c["Hkv"], page, c["dh"])
            s["v_pages"] = _normal(g, c["L"], N, c["Hkv"], page, c["dh"])
        else:
            width = max(_pages(p + c["T"], page) for p in ln)
        s["block_table"] = _scattered_table(g, counts, width, N)
        s["n_pages"] = _i32(counts)
        held = s["block_table"].flatten()
        s["refcount"] = torch.zeros(N, dtype=torch.int32, device=DEV)
        s["refcount"][held[held >= 0].long()] = 1
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import medusa_draft_heads_b200 as md
    c = case
    s["md"] = md
    if c["op"] in ("attention", "commit"):
        s["tree"] = md.Tree(s["parent"], s["rank"], KPH)
    if c["op"] == "attention":
        dt = torch.float32 if c["out"] == "fp32" else torch.bfloat16
        s["out"] = torch.empty(s["q"].shape, dtype=dt, device=DEV)
        s["ws"] = md.workspace(md.attention_paged_workspace_bytes(c["B"], c["T"], c["Hq"], c["Hkv"], c["dh"], c["page"],
                                                                  s["block_table"].shape[1]))
    elif c["op"] == "rope":
        s["q_out"] = torch.zeros((c["B"], c["T"], c["Hq"], c["dh"]), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "commit":
        for k in ("new_prefix_len", "next_root", "next_head_row"):
            s[k] = torch.empty_like(s["prefix_len"])
    elif c["op"] == "fork":
        s["ws"] = md.workspace(md.pages_fork_workspace_bytes(c["B"], c["n"]))
    else:
        s["held"] = torch.empty_like(s["block_table"])
    return s


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"attention": _plain_attention, "rope": _plain_rope, "commit": _plain_commit, "resize": _plain_resize,
            "fork": _plain_fork}[c["op"]](state, c)


def _run_own(s, c):
    md = s["md"]
    if c["op"] == "attention":
        md.tree_attention_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["prefix_len"], s["tree"], s["out"],
                                s["ws"])
        return s["out"]
    if c["op"] == "rope":
        md.qk_rope_append(s["q"], s["k"], s["v"], s["pos"], s["inv_freq"], s["q_out"], s["k_pages"], s["v_pages"],
                          s["block_table"], s["prefix_len"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6,
                          interleaved=c["pairs"] == "adjacent", n_new=s["n_new"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["op"] == "commit":
        md.tree_commit_paged(s["k_pages"], s["v_pages"], s["block_table"], s["tree"], s["prefix_len"], s["accept_len"],
                             s["path"], s["bonus"], s["new_prefix_len"], s["next_root"], s["next_head_row"])
        return {k: s[k] for k in ("k_pages", "v_pages", "new_prefix_len", "next_root", "next_head_row")}
    if c["op"] == "resize":
        md.pages_resize(s["block_table"], s["n_pages"], s["refcount"], s["prefix_len"], c["page"], extra=c["T"])
        s["held"].copy_(s["block_table"])          # what the step between the two calls reads
        md.pages_resize(s["block_table"], s["n_pages"], s["refcount"], s["prefix_len"], c["page"])
        return {k: s[k] for k in ("held", "block_table", "n_pages", "refcount")}
    md.pages_fork(s["k_pages"], s["v_pages"], s["block_table"], s["n_pages"], s["refcount"], s["src"], s["dst"],
                  s["prefix_len"], s["ws"])
    return {k: s[k] for k in ("k_pages", "v_pages", "block_table", "n_pages", "refcount", "prefix_len")}


# -------------------------------------------------------------- plain forms

def _plain_attention(s, c):
    T, Hkv, dh, G = c["T"], c["Hkv"], c["dh"], c["Hq"] // c["Hkv"]
    hide = s["hide"].repeat_interleave(G, dim=0)                        # [T*G, T]
    outs = []
    for b, P in enumerate(s["lens"]):
        n = P + T
        pages = s["block_table"][b, :_pages(n, c["page"])].long()
        k = s["k_pages"][pages].transpose(0, 1).reshape(Hkv, -1, dh)[:, :n].float()
        v = s["v_pages"][pages].transpose(0, 1).reshape(Hkv, -1, dh)[:, :n].float()
        q = s["q"][b].view(T, Hkv, G, dh).transpose(0, 1).reshape(Hkv, T * G, dh).float()
        x = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(dh))
        x[:, :, P:].masked_fill_(hide, float("-inf"))
        x = torch.exp(x - x.amax(dim=-1, keepdim=True))
        o = torch.matmul(x, v) / x.sum(dim=-1, keepdim=True)
        outs.append(o.view(Hkv, T, G, dh).transpose(0, 1).reshape(T, c["Hq"], dh))
    out = torch.stack(outs)
    return out if c["out"] == "fp32" else out.bfloat16()


def _plain_rope(s, c):
    if "q_out" not in s:
        s["q_out"] = torch.zeros((c["B"], c["T"], c["Hq"], c["dh"]), dtype=torch.bfloat16, device=DEV)
    ang = s["pos"].double()[..., None] * s["inv_freq"].double()          # [B, T, rot/2]
    cos, sin = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    half = c["rot"] // 2

    def norm_rotate(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * w.float()
        y = x.clone()
        if c["pairs"] == "half":
            a, b = x[..., :half], x[..., half:2 * half]
            y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
        return y.bfloat16()

    qr, kr = norm_rotate(s["q"], s["q_norm"]), norm_rotate(s["k"], s["k_norm"])
    for b, n in enumerate(s["new_list"]):
        s["q_out"][b, :n] = qr[b, :n]
        slots = s["lens"][b] + torch.arange(n, device=DEV)
        page, row = s["block_table"][b, slots // c["page"]].long(), slots % c["page"]
        s["k_pages"][page, :, row] = kr[b, :n]
        s["v_pages"][page, :, row] = s["v"][b, :n]
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_commit(s, c):
    K = s["path"].shape[1] - 1
    live = torch.arange(K + 1, device=DEV)[None] <= s["accept_len"][:, None]
    P = s["prefix_len"][:, None]
    to = P + torch.arange(K + 1, dtype=torch.int32, device=DEV)[None]
    frm = torch.where(live, P + s["path"], P)
    to = torch.where(live, to, P)                       # what is not on the path copies the root onto itself
    rows = torch.arange(c["B"], device=DEV)[:, None]
    fp, fr = s["block_table"][rows, frm // c["page"]].long(), frm.long() % c["page"]
    tp, tr = s["block_table"][rows, to // c["page"]].long(), to.long() % c["page"]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, tp, :, tr] = pool[:, fp, :, fr]
    last = s["path"].gather(1, s["accept_len"][:, None].long())[:, 0]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "new_prefix_len": s["prefix_len"] + s["accept_len"] + 1,
            "next_root": s["bonus"].clone(),
            "next_head_row": torch.arange(c["B"], dtype=torch.int32, device=DEV) * c["T"] + last}


def _lowest_free(refcount):
    """The free pages' ids in ascending order (then the others'), and how many are free."""
    taken = (refcount != 0).to(torch.int32)
    return torch.argsort(taken, stable=True).to(torch.int32), (1 - taken).sum()


def _resize(table, n_pages, refcount, length, page, extra):
    idx = torch.arange(table.shape[1], dtype=torch.int32, device=DEV)[None]
    want = torch.where(length < 0, 0, (length + extra + page - 1) // page)
    drop = (idx >= want[:, None]) & (idx < n_pages[:, None])
    refcount.index_add_(0, torch.where(drop, table, 0).flatten().long(), -drop.flatten().to(torch.int32))
    table.copy_(torch.where(drop, -1, table))
    n_pages.copy_(torch.minimum(n_pages, want))
    need = want - n_pages
    order, free = _lowest_free(refcount)
    upto = torch.cumsum(need, 0)
    need = torch.where(upto <= free, need, 0)
    grow = (idx >= n_pages[:, None]) & (idx < (n_pages + need)[:, None])
    which = torch.where(grow, (upto - need)[:, None] + idx - n_pages[:, None], 0)
    got = order[which.long()]
    table.copy_(torch.where(grow, got, table))
    refcount.index_add_(0, torch.where(grow, got, 0).flatten().long(), grow.flatten().to(torch.int32))
    n_pages.add_(need.to(torch.int32))


def _plain_resize(s, c):
    _resize(s["block_table"], s["n_pages"], s["refcount"], s["prefix_len"], c["page"], c["T"])
    held = s["block_table"].clone()
    _resize(s["block_table"], s["n_pages"], s["refcount"], s["prefix_len"], c["page"], 0)
    return {"held": held, "block_table": s["block_table"], "n_pages": s["n_pages"], "refcount": s["refcount"]}


def _plain_fork(s, c):
    table, n_pages, ref, ps = s["block_table"], s["n_pages"], s["refcount"], c["page"]
    src, dst = s["src"].long(), s["dst"].long()
    idx = torch.arange(table.shape[1], dtype=torch.int32, device=DEV)[None]
    old = idx < n_pages[dst][:, None]
    ref.index_add_(0, torch.where(old, table[dst], 0).flatten().long(), -old.flatten().to(torch.int32))
    ln = s["prefix_len"][src]
    full, part = ln // ps, ln % ps
    need = (part > 0).to(torch.int32)
    order, _ = _lowest_free(ref)
    fresh = order[(torch.cumsum(need, 0) - need).long()]
    shared = idx < full[:, None]
    new = torch.where(shared, table[src], -1)
    last = (idx == full[:, None]) & (need[:, None] > 0)
    new = torch.where(last, fresh[:, None], new)
    ref.index_add_(0, torch.where(shared, new, 0).flatten().long(), shared.flatten().to(torch.int32))
    ref.index_add_(0, fresh.long(), need)
    for i, (a, b) in enumerate(zip(s["src_list"], s["dst_list"])):
        n = s["lens"][a] % ps
        if n:
            f, t = table[a, s["lens"][a] // ps].long(), fresh[i].long()
            for pool in (s["k_pages"], s["v_pages"]):
                pool.index_copy_(1, t[None], torch.cat((pool.index_select(1, f[None])[:, :, :, :n],
                                                        pool.index_select(1, t[None])[:, :, :, n:]), dim=3))
    table[dst] = new
    n_pages[dst] = full + need
    s["prefix_len"][dst] = ln
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "block_table": table, "n_pages": n_pages, "refcount": ref,
            "prefix_len": s["prefix_len"]}


# ------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """Attention and rotation in 64 bits; moves and page numbers are no computed numbers."""
    c = case
    if c["op"] not in ("attention", "rope"):
        return None
    s = _inputs(c, seed)
    page = c["page"]
    if c["op"] == "attention":
        T, G = c["T"], c["Hq"] // c["Hkv"]
        out = torch.empty((c["B"], T, c["Hq"], c["dh"]), dtype=torch.float64, device=DEV)
        bias = torch.full((T, T), -math.inf, dtype=torch.float64)
        for t in range(T):
            bias[t, t] = 0.0
            if s["parent"][t] >= 0:
                bias[t] = torch.maximum(bias[t], bias[s["parent"][t]])
        bias = bias.to(DEV)
        for b, P in enumerate(s["lens"]):
            slots = torch.arange(P + T, device=DEV)
            pg, row = s["block_table"][b].long()[slots // page], slots % page
            for g in range(c["Hkv"]):
                k, v = s["k_pages"][pg, g, row].double(), s["v_pages"][pg, g, row].double()
                for h in range(g * G, (g + 1) * G):
                    x = s["q"][b, :, h].double() @ k.T / math.sqrt(c["dh"])
                    x[:, P:] += bias
                    w = torch.exp(x - torch.logsumexp(x, dim=1)[:, None])
                    out[b, :, h] = w @ v
        return out
    half = c["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["pos"].double()[..., None] * s["inv_freq"].double())

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["dh"] + 1e-6) * w.double()
        head, rest = x[..., :2 * half], x[..., 2 * half:]
        if c["pairs"] == "half":
            z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn[:, :, None]
            return torch.cat((z.real, z.imag, rest), dim=-1)
        z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) * turn[:, :, None]
        return torch.cat((torch.view_as_real(z).flatten(-2), rest), dim=-1)

    q = torch.zeros((c["B"], c["T"], c["Hq"], c["dh"]), dtype=torch.float64, device=DEV)
    kp = s["k_pages"].double()
    qr, kr = rotated(s["q"], s["q_norm"]), rotated(s["k"], s["k_norm"])
    for b, (P, n) in enumerate(zip(s["lens"], s["new_list"])):
        q[b, :n] = qr[b, :n]
        for i, pg in enumerate(s["block_table"][b].tolist()):
            lo, hi = max(P, i * page), min(P + n, (i + 1) * page)
            if lo < hi:
                kp[pg, :, lo - i * page:hi - i * page] = kr[b, lo - P:hi - P].transpose(0, 1)
    return {"q": q, "k_pages": kp, "v_pages": None}
