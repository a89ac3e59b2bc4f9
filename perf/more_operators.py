"""Cases of rotary positions, of appending to a paged KV cache, and of attention for trees of drafted tokens over it.

A paged cache is a buffer of KV rows [rows, Hkv, d] (bf16, or e4m3 codes with a power-of-two scale per row and head): key j
of request b lies at row page_table[b, j // page] * page + j % page.  Request b has kv_lens[b] cached keys; its new tokens
(the nodes of its tree) are the query rows q_start[b] .. q_start[b + 1] - 1 and follow as keys kv_lens[b], kv_lens[b] + 1 ...

- ``rope``: Q and K rows are rotated: pair c of a row by the angle positions[axis(c)] * inv_freq[c] (``inverse``: back, which
  is the gradient).  Pairs are columns (c, c + pairs), or (2c, 2c + 1) where interleaved.
- ``append``: new K rows are rotated and stored with V at given cache rows (a negative one is padding), and Q is rotated.
- ``layout``: a step's cache rows and positions, and each node's ancestors as bits, from the nodes' parents.
- ``attn``: node i of a request attends to the request's cached keys and to the nodes in its mask (without masks: to the
  nodes up to itself).

``run`` computes them from elementary operations, or, where ``own`` is true, calls the library.
"""

import math
import random

import torch

own = False


def listed():
    return [
        # an image and video prompt: positions of time, height and width; 8192 tokens
        dict(name="rope_video", op="rope", n=8192, Hq=32, Hkv=8, d=128, pairs=64, axes=3, interleaved=False, inverse=False,
             dtype="bf16"),
        # the gradient of a short odd batch, interleaved pairs, half of the columns, fp32
        dict(name="rope_grad", op="rope", n=1001, Hq=12, Hkv=4, d=64, pairs=16, axes=1, interleaved=True, inverse=True,
             dtype="fp32"),
        # one decode step of 64 requests: latency
        dict(name="append_step", op="append", n=64, Hq=32, Hkv=8, d=128, dv=128, pairs=64, axes=1, kv="bf16", padded=False),
        # a prefill chunk into a quantised cache, padded, positions of three axes
        dict(name="append_chunk_e4m3", op="append", n=4096, Hq=32, Hkv=8, d=128, dv=128, pairs=64, axes=3, kv="e4m3",
             padded=True),
        # latent rows (absorbed form: one head of 576 whose last 64 columns are rotated, no V of its own)
        dict(name="append_latent", op="append", n=16384, Hq=0, Hkv=1, d=576, dv=0, pairs=32, axes=1, kv="bf16",
             padded=False),
        # one request's drafted chain: latency
        dict(name="layout_one", op="layout", B=1, T=8, kv_max=2000, page=16, lens=1),
        # the trees of a serving batch
        dict(name="layout_batch", op="layout", B=256, T=64, kv_max=8192, page=16, lens=2),
        # one token over a short cache: latency
        dict(name="attn_one", op="attn", kv="bf16", B=1, T=1, tree=False, Hq=32, Hkv=8, d=128, kv_max=1000, page=16, lens=3),
        # a decode step of a serving batch on a quantised cache
        dict(name="attn_decode_e4m3", op="attn", kv="e4m3", B=64, T=1, tree=False, Hq=32, Hkv=8, d=128, kv_max=8192, page=64,
             lens=4),
        # drafted chains of up to 8 tokens being verified, pages of 16
        dict(name="attn_chain", op="attn", kv="bf16", B=16, T=8, tree=False, Hq=32, Hkv=8, d=128, kv_max=8192, page=16,
             lens=5),
        # trees of up to 26 nodes, d = 64, quantised, ragged
        dict(name="attn_tree_d64_e4m3", op="attn", kv="e4m3", B=13, T=26, tree=True, Hq=16, Hkv=2, d=64, kv_max=4001, page=32,
             lens=6),
        # the largest: trees of up to 64 nodes over long caches
        dict(name="attn_tree_large", op="attn", kv="bf16", B=32, T=64, tree=True, Hq=32, Hkv=8, d=128, kv_max=16384, page=16,
             lens=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "layout", "attn", "attn", "attn"])
    if op == "rope":
        d, pairs = rng.choice([(64, 32), (64, 16), (128, 64), (128, 64), (96, 48), (256, 128), (80, 16)])
        Hq, Hkv = rng.choice([(8, 8), (32, 8), (16, 2), (12, 4), (7, 1)])
        return dict(op=op, n=_log_int(rng, 1, 8192), Hq=Hq, Hkv=Hkv, d=d, pairs=pairs, axes=rng.choice([1, 2, 3]),
                    interleaved=rng.random() < 0.4, inverse=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "append":
        Hq, Hkv, d, dv, pairs = rng.choice([(32, 8, 128, 128, 64), (32, 8, 128, 128, 64), (8, 8, 64, 64, 32), (16, 2, 128, 64, 32),
                                            (0, 4, 96, 96, 48), (0, 1, 576, 0, 32), (12, 4, 256, 256, 32)])
        return dict(op=op, n=_log_int(rng, 1, 8192), Hq=Hq, Hkv=Hkv, d=d, dv=dv, pairs=pairs, axes=rng.choice([1, 1, 3]),
                    kv=rng.choice(["bf16", "e4m3"]), padded=rng.random() < 0.5)
    page = rng.choice([16, 16, 32, 64, 128, 256])
    if op == "layout":
        return dict(op=op, B=_log_int(rng, 1, 256), T=_log_int(rng, 1, 64), kv_max=_log_int(rng, 1, 16384), page=page,
                    lens=rng.randrange(1 << 20))
    most = work(listed()[-1])
    while True:
        Hq, Hkv = rng.choice([(8, 8), (32, 8), (32, 8), (16, 2), (12, 4), (40, 8), (64, 8), (32, 1), (7, 1)])
        c = dict(op="attn", kv=rng.choice(["bf16", "e4m3"]), B=_log_int(rng, 1, 128), T=_log_int(rng, 1, 64),
                 tree=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, d=rng.choice([64, 128, 128]), kv_max=_log_int(rng, 1, 16384),
                 page=page, lens=rng.randrange(1 << 20))
        w = work(c)
        keys = c["B"] * (c["kv_max"] + c["T"])
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and keys * c["Hkv"] * c["d"] <= 1 << 30 and \
                keys * c["Hq"] * c["T"] <= 1 << 31:
            return c


def _lens(case):
    """Nodes, cached keys and parents of each request's nodes (a root has -1), from the case alone.  A few requests of a
    large batch have an empty cache, or no nodes (free slots of a padded batch)."""
    rng = random.Random(case["lens"])
    nodes, kv, parents = [], [], []
    for b in range(case["B"]):
        t = rng.randint(max(1, case["T"] // 2), case["T"])
        if b % 31 == 30:
            t = 0
        nodes.append(t)
        kv.append(0 if b % 29 == 28 else rng.randint((case["kv_max"] + 3) // 4, case["kv_max"]))
        for i in range(t):
            chain = case["op"] == "attn" and not case["tree"]
            # a tree's nodes hang below one of the last few, so that it has some depth
            parents.append(i - 1 if chain else rng.randint(max(-1, i - 7), i - 1))
    return nodes, kv, parents


def _depths(nodes, parents):
    d, at = [], 0
    for t in nodes:
        for i in range(t):
            p = parents[at + i]
            d.append(0 if p < 0 else d[at + p] + 1)
        at += t
    return d


def _padding(case):
    """Rows of a padded append that are padding: every 16th and the last."""
    return [i for i in range(case["n"]) if case["padded"] and (i % 16 == 15 or i == case["n"] - 1)]


def work(case):
    op = case["op"]
    if op == "rope":
        x = 2 if case["dtype"] == "bf16" else 4
        values = case["n"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": 2 * x * values + 4 * case["n"] * case["axes"],
                "flops": 6 * case["n"] * (case["Hq"] + case["Hkv"]) * case["pairs"]}
    if op == "append":
        n, kept = case["n"], case["n"] - len(_padding(case))
        vectors = case["Hkv"] * (2 if case["dv"] else 1)
        values = case["Hkv"] * (case["d"] + case["dv"])
        out = 2 * values if case["kv"] == "bf16" else values + 4 * vectors
        return {"bytes": n * case["Hq"] * case["d"] * 4 + kept * (2 * values + out) + 4 * n * (case["axes"] + 1),
                "flops": 6 * (n * case["Hq"] + kept * case["Hkv"]) * case["pairs"]}
    nodes, kv, parents = _lens(case)
    N, B = sum(nodes), case["B"]
    words = -(-case["T"] // 32)
    pages = sum(-(-(t + k) // case["page"]) for t, k in zip(nodes, kv))
    if op == "layout":
        # parents, lengths and the nodes' pages in; rows, positions and masks out
        pages = sum((t + k - 1) // case["page"] - k // case["page"] + 1 for t, k in zip(nodes, kv) if t)
        return {"bytes": 4 * (N + 2 * B + pages + N * (2 + words)), "flops": sum(_depths(nodes, parents))}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    row = Hkv * 2 * (2 * d if case["kv"] == "bf16" else d + 4)
    visible = sum(t * k for t, k in zip(nodes, kv)) + sum(_depths(nodes, parents)) + N
    keys = sum(t + k for t, k in zip(nodes, kv) if t)
    return {"bytes": keys * row + N * Hq * (4 * d + 4) + 4 * (pages + 2 * B + (N * words if case["tree"] else 0)),
            "flops": 4 * d * Hq * visible}


# ----------------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _keys(g, shape, dtype=torch.bfloat16):
    """Keys as projections make them: a few channels much larger than the others."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.05
    return (x * torch.where(loud, 4.0, 0.8)).to(dtype)


def _rotation(case, g, s):
    """Frequencies, the axis of each pair (the axes take turns) and the positions of the rows."""
    pairs, A = case["pairs"], case["axes"]
    s["inv_freq"] = 500000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    s["axis"] = torch.arange(pairs) % A
    first = torch.randint(0, 1 << 20, (A, 1), generator=g, device="cuda")
    s["positions"] = (first + torch.randint(0, 4096, (A, case["n"]), generator=g, device="cuda")).to(torch.int32)
    s["first"] = case["d"] - 2 * pairs if case["Hkv"] == 1 and case["d"] == 576 else 0
    s["angle"] = (s["inv_freq"].cuda(), s["axis"].cuda())
    if own:
        import context_causal_attention_cp_gb300 as cpa

        s["rope"] = cpa.make_rope(s["inv_freq"], axes=s["axis"], first=s["first"], interleaved=case.get("interleaved", False))


def _pages(case, g, nodes, kv, s):
    """A page table whose pages lie anywhere in the cache; entries behind a request's last page are -1."""
    page = case["page"]
    need = [-(-(t + k) // page) for t, k in zip(nodes, kv)]
    total = sum(need) + max(4, sum(need) // 8)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["B"], max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    count = torch.tensor(need, device="cuda")
    at = torch.arange(table.shape[1], device="cuda")
    first = torch.cumsum(count, 0) - count
    held = at < count[:, None]
    table[held] = order[(first[:, None] + at)[held]]
    s["page_table"], s["rows"] = table, total * page
    s["q_start"] = torch.tensor([0] + nodes, device="cuda").cumsum(0).to(torch.int32)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op in ("rope", "append"):
        n, Hq, Hkv, d = case["n"], case["Hq"], case["Hkv"], case["d"]
        _rotation(case, g, s)
        dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
        s["q"], s["k"] = _normal(g, (n, Hq, d), dtype) if Hq else None, _keys(g, (n, Hkv, d), dtype)
        s["out_q"] = torch.empty_like(s["q"]) if Hq else None
        if op == "rope":
            s["out_k"] = torch.empty_like(s["k"])
            return s
        dv = case["dv"]
        s["v"] = _normal(g, (n, Hkv, dv)) if dv else None
        rows = n + n // 2 + 5
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32)
        if _padding(case):
            s["slots"][torch.tensor(_padding(case), device="cuda")] = -1
        # what the cache holds before
        s["k_cache"], s["v_cache"] = _keys(g, (rows, Hkv, d)), _normal(g, (rows, Hkv, dv)) if dv else None
        s["k_scale"] = s["v_scale"] = None
        if case["kv"] == "e4m3":
            s["k_cache"], s["k_scale"] = _quantize(s["k_cache"])
            if dv:
                s["v_cache"], s["v_scale"] = _quantize(s["v_cache"])
        if own:
            import context_causal_attention_cp_gb300 as cpa

            s["cache"] = cpa.KVCache(s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]) if case["kv"] == "e4m3" else \
                (s["k_cache"], s["v_cache"])
        return s
    nodes, kv, parents = _lens(case)
    N = sum(nodes)
    _pages(case, g, nodes, kv, s)
    s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    s["words"] = -(-case["T"] // 32)
    if op == "layout":
        if N:  # another seed, other trees: some nodes become roots
            cut = torch.rand(N, generator=g, device="cuda") < 0.1
            s["parents"][cut] = -1
        s["slots"], s["positions"] = (torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(2))
        s["mask"] = torch.empty((N, s["words"]), dtype=torch.int32, device="cuda")
        return s
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    s.update(q=_normal(g, (N, Hq, d)), scale=d ** -0.5, k=_keys(g, (s["rows"], Hkv, d)), v=_normal(g, (s["rows"], Hkv, d)),
             k_scale=None, v_scale=None, mask=None, out=torch.empty((N, Hq, d), dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty((N, Hq), dtype=torch.float32, device="cuda"))
    if case["tree"]:  # made once a step, used by every layer
        s["mask"] = _layout(s)["mask"]
    if case["kv"] == "e4m3":
        (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = _quantize(s["k"]), _quantize(s["v"])
    if own:
        import context_causal_attention_cp_gb300 as cpa

        s["workspace"] = cpa.alloc_tree_workspace(Hq, Hkv, d, case["T"])
    return s


# ------------------------------------------------------------------ plain forms --
def _quantize(x):
    """Codes [rows, Hkv, d] and scales [Hkv, rows] of the rows x."""
    x = x.float()
    a = x.abs()
    a = torch.where(a < math.inf, a, 0.0).amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e with m in [1/2, 1), and 448 = 7/8 2^9
    e = torch.where(a > 0, e - 9 + (m > 0.875).to(e.dtype), -117).clamp(-117, 119)
    scale = torch.ldexp(torch.ones_like(a), e)
    y = x * torch.ldexp(torch.ones_like(a), -e)[..., None]
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), scale.t().contiguous()


def _turn(s):
    """cos and sin [n, 1, pairs] of the rows' angles: the angles of far positions need 64 bits."""
    inv_freq, axis = s["angle"]
    a = s["positions"][axis].t().double() * inv_freq
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, turn, first, pairs, interleaved, inverse):
    """x in fp32, rotated."""
    cos, sin = turn
    sin = -sin if inverse else sin
    y = x.float().clone()
    r = y[..., first:first + 2 * pairs]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :pairs], r[..., pairs:])
    u, w = a * cos - b * sin, b * cos + a * sin
    a.copy_(u)
    b.copy_(w)
    return y


def _rope(s):
    case, turn = s["case"], _turn(s)
    args = turn, s["first"], case["pairs"], case["interleaved"], case["inverse"]
    return {"q": _rotate(s["q"], *args).to(s["q"].dtype), "k": _rotate(s["k"], *args).to(s["k"].dtype)}


def _append(s):
    case, turn = s["case"], _turn(s)
    args = turn, s["first"], case["pairs"], False, False
    kept = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"][kept].long()
    for name, x in (("k", _rotate(s["k"], *args)), ("v", s["v"])):
        if x is None:
            continue
        cache, scales = s[name + "_cache"], s[name + "_scale"]
        if scales is None:
            cache[at] = x[kept].to(cache.dtype)
        else:
            codes, sc = _quantize(x)
            cache.view(torch.uint8)[at] = codes.view(torch.uint8)[kept]
            scales[:, at] = sc[:, kept]
    q = _rotate(s["q"], *args).to(s["q"].dtype) if s["q"] is not None else None
    return {"q": q, "k": s["k_cache"], "k_scale": s["k_scale"], "v": s["v_cache"], "v_scale": s["v_scale"]}


def _nodes(s):
    """Request and number within it of each node."""
    count = (s["q_start"][1:] - s["q_start"][:-1]).long()
    N = s["parents"].shape[0]
    req = torch.repeat_interleave(torch.arange(count.shape[0], device="cuda"), count, output_size=N)
    return req, torch.arange(N, device="cuda") - s["q_start"][req].long()


def _layout(s):
    case = s["case"]
    B, T, page = case["B"], case["T"], case["page"]
    req, i = _nodes(s)
    at = s["kv_lens"][req].long() + i
    slots = s["page_table"][req, at // page] * page + at % page
    # ancestors: the closure of the parent relation, by squaring
    up = torch.zeros((B, T, T + 1), device="cuda")
    up[req, i, s["parents"].long()] = 1.0  # (a root's -1 is the last column, which is dropped)
    up = up[..., :T]
    up[req, i, i] = 1.0
    for _ in range(max(1, (T - 1).bit_length())):
        up = (up @ up).clamp_(max=1.0)
    seen = up[req, i].long()
    positions = s["kv_lens"][req].long() + seen.sum(-1) - 1
    seen = torch.cat([seen, seen.new_zeros(seen.shape[0], 32 * s["words"] - T)], 1).view(-1, s["words"], 32)
    mask = (seen << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask)
    return {"slots": slots.to(torch.int32), "positions": positions.to(torch.int32), "mask": mask.to(torch.int32)}


def _values(codes, scales, rows):
    if scales is None:
        return codes[rows].float()
    return codes.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float() * scales[:, rows].t()[..., None]


def _attend(s):
    case, q = s["case"], s["q"].float()
    N, Hq, d = q.shape
    B, T, Hkv, page = case["B"], case["T"], case["Hkv"], case["page"]
    g, K = Hq // Hkv, case["kv_max"] + T
    req, i = _nodes(s)
    x = q.new_zeros((B, T, Hq, d))
    x[req, i] = q
    x = x.view(B, T, Hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * g, d)
    key = torch.arange(K, device="cuda")
    rows = s["page_table"][:, (key // page).clamp(max=s["page_table"].shape[1] - 1)].long().clamp(min=0) * page + key % page
    k, v = (_values(s[name], s[name + "_scale"], rows.reshape(-1)).view(B, K, Hkv, d).permute(0, 2, 1, 3) for name in "kv")
    # keys that a node sees: the cached ones, and nodes by its mask
    node = key - s["kv_lens"].long()[:, None]
    if s["mask"] is None:
        seen = node[:, None, :] <= torch.arange(T, device="cuda")[:, None]
    else:
        mask = s["mask"].new_zeros((B, T, s["words"]))
        mask[req, i] = s["mask"]
        at = node.clamp(0, 32 * s["words"] - 1)
        bits = torch.gather(mask, 2, (at // 32)[:, None].expand(B, T, K)) >> (at % 32)[:, None]
        seen = (node < 0)[:, None] | (((bits & 1) > 0) & (node < 32 * s["words"])[:, None])
    p = (x @ k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, T, g, K)
    p.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = p.amax(-1)
    m = torch.where(m > -math.inf, m, 0.0)
    p.sub_(m[..., None]).exp_()
    total = p.sum(-1)
    o = (p.view(B, Hkv, T * g, K) @ v).view(B, Hkv, T, g, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d)[req, i]
    lse = (m + total.log()).permute(0, 2, 1, 3).reshape(B, T, Hq)[req, i]
    return {"o": o.to(torch.bfloat16), "lse": lse}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _rope, "append": _append, "layout": _layout, "attn": _attend}[op](s)
    import context_causal_attention_cp_gb300 as cpa

    if op == "rope":
        q, k = cpa.cp_rope(s["rope"], s["q"], s["k"], s["positions"], inverse=s["case"]["inverse"], out_q=s["out_q"],
                           out_k=s["out_k"])
        return {"q": q, "k": k}
    if op == "append":
        q = cpa.cp_kv_append(s["cache"], s["k"], s["v"], s["slots"], rope=s["rope"], positions=s["positions"], q=s["q"],
                             out_q=s["out_q"])
        return {"q": q, "k": s["k_cache"], "k_scale": s["k_scale"], "v": s["v_cache"], "v_scale": s["v_scale"]}
    if op == "layout":
        slots, positions, mask = cpa.cp_tree_layout(s["q_start"], s["kv_lens"], s["page_table"], s["case"]["page"],
                                                    s["parents"].shape[0], parents=s["parents"], slots=s["slots"],
                                                    positions=s["positions"], mask=s["mask"])
        return {"slots": slots, "positions": positions, "mask": mask}
    o, lse, _ = cpa.cp_attn_tree(s["q"], s["k"], s["v"], s["page_table"], s["case"]["page"], s["q_start"], s["kv_lens"],
                                 s["scale"], mask=s["mask"], max_nodes=s["case"]["T"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------ exact --
def _exact_codes(x):
    """The definition in 64 bits: (code values [rows, Hkv, d], scales [Hkv, rows])."""
    a = torch.nan_to_num(x.abs(), nan=0.0, posinf=0.0).amax(-1)
    e = torch.ceil(torch.log2(a / 448.0))
    e = e + (a > 448.0 * torch.exp2(e)).double() - (a <= 448.0 * torch.exp2(e - 1)).double()
    e = torch.where(a > 0, e, -117.0).clamp(-117.0, 119.0)
    y = (x / torch.exp2(e)[..., None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.exp2(e).t()


def _exact_rotate(s, x):
    """The pairs as complex numbers, times exp(i angle)."""
    case = s["case"]
    pairs, lo = case["pairs"], s["first"]
    inv_freq, axis = s["angle"]
    angle = torch.stack([s["positions"][int(axis[c])].double() * inv_freq[c] for c in range(pairs)], 1)
    if case.get("inverse"):
        angle = -angle
    y = x.double().clone()
    part = y[..., lo:lo + 2 * pairs]
    pick = torch.arange(pairs, device="cuda")
    re, im = (2 * pick, 2 * pick + 1) if case.get("interleaved") else (pick, pairs + pick)
    z = torch.complex(part[..., re], part[..., im]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y[..., lo + re], y[..., lo + im] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _exact_rotate(s, s["q"]), "k": _exact_rotate(s, s["k"])}
    if case["op"] == "append":
        out = {"q": None if s["q"] is None else _exact_rotate(s, s["q"])}
        kept = s["slots"] >= 0
        at = s["slots"][kept].long()
        for name in ("k", "v"):
            out[name] = out[name + "_scale"] = None
            if s[name] is None:
                continue
            new = (_exact_rotate(s, s["k"]) if name == "k" else s["v"].double())[kept]
            cache = s[name + "_cache"].double()
            if s[name + "_scale"] is not None:
                new, sc = _exact_codes(new)
                out[name + "_scale"] = s[name + "_scale"].double()
                out[name + "_scale"][:, at] = sc
            cache[at] = new
            out[name] = cache
        return out
    if case["op"] == "layout":
        return None  # whole numbers
    nodes, kv, parents = _lens(case)
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    g = Hq // Hkv
    os, ls, n0 = [], [], 0
    for b, (t, held) in enumerate(zip(nodes, kv)):
        if not t:
            continue
        key = torch.arange(held + t, device="cuda")
        rows = s["page_table"][b][key // page].long() * page + key % page

        def values(name):
            x = s[name].view(torch.uint8)[rows].view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else s[name][rows]
            x = x.double()
            return (x if s[name + "_scale"] is None else x * s[name + "_scale"][:, rows].double().t()[..., None]).transpose(0, 1)

        sees = torch.zeros((t, t), dtype=torch.bool)
        for i in range(t):
            j = i
            while j >= 0:
                sees[i, j] = True
                j = parents[n0 + j]
        sees = torch.cat([torch.ones((t, held), dtype=torch.bool), sees], 1).cuda()
        q = s["q"][n0:n0 + t].double().view(t, Hkv, g, d).permute(1, 2, 0, 3).reshape(Hkv, g * t, d)
        x = (q @ values("k").transpose(1, 2)).view(Hkv, g, t, held + t) * s["scale"]
        x = x.masked_fill(~sees, -math.inf)
        lse = torch.logsumexp(x, -1)
        o = (torch.exp(x - lse[..., None]).view(Hkv, g * t, held + t) @ values("v")).view(Hkv, g, t, d)
        os.append(o.permute(2, 0, 1, 3).reshape(t, Hq, d))
        ls.append(lse.permute(2, 0, 1).reshape(t, Hq))
        n0 += t
    return {"o": torch.cat(os) if os else s["q"].double(), "lse": torch.cat(ls) if ls else s["lse"].double()}
