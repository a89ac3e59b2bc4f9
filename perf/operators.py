"""Cases of the quantised KV cache and of attention over a shared prefix.

Three operators, all over a KV buffer of rows [rows, Hkv, d]:

- ``write``: new K and V rows are quantised to e4m3 with one power-of-two scale per row and KV head, and stored at given
  cache rows (a negative slot is padding).  With a = max finite |x|, e = clamp(ceil(log2(a / 448)), -117, 119):
  scale = 2^e, code = e4m3(x / scale), rounded to nearest even and saturated.
- ``read``: cache rows given by an index are read back as code * scale.
- ``attn``: every request of a batch attends to one shared prefix and to its own causal keys behind it.  The buffer is
  bf16, or the quantised cache.

``run`` computes them from elementary operations, or, where ``own`` is true, calls the library.
"""

import math
import random

import torch

own = False

PAGE = 16  # read: the index is made of runs of this many rows, as a paged allocator hands them out


def listed():
    return [
        # one decode step's new K and V of 64 requests: latency
        dict(name="write_step", op="write", n=64, Hkv=8, d=128, dv=128, dtype="bf16", padded=False),
        # a prefill chunk whose batch is padded
        dict(name="write_chunk", op="write", n=8192, Hkv=8, d=128, dv=128, dtype="bf16", padded=True),
        # the latent rows of a 16K prompt (absorbed form: one head of 576, no V of its own)
        dict(name="write_latent", op="write", n=16384, Hkv=1, d=576, dv=0, dtype="bf16", padded=False),
        # a cached 32K prefix read back as the gathered KV of a prefill
        dict(name="read_prefix", op="read", n=32768, Hkv=8, d=128, dv=128, dtype="bf16"),
        # a short odd run at d = 64, in fp32
        dict(name="read_short", op="read", n=777, Hkv=8, d=64, dv=64, dtype="fp32"),
        # one token behind a short prefix: latency
        dict(name="attn_one", op="attn", kv="bf16", B=1, q_max=1, Hq=32, Hkv=8, d=128, prefix=1024, own_max=100, lens=1),
        # a small batch on a quantised cache
        dict(name="attn_small_e4m3", op="attn", kv="e4m3", B=8, q_max=1, Hq=32, Hkv=8, d=128, prefix=8192, own_max=512,
             lens=2),
        # 64 decode queries over 65536 shared keys
        dict(name="attn_64k", op="attn", kv="bf16", B=64, q_max=1, Hq=32, Hkv=8, d=128, prefix=65536, own_max=128, lens=3),
        # a serving batch on a quantised cache, own turns of up to 2048 tokens
        dict(name="attn_serve_e4m3", op="attn", kv="e4m3", B=64, q_max=1, Hq=32, Hkv=8, d=128, prefix=32768, own_max=2048,
             lens=4),
        # drafted tokens being verified: up to 8 queries a request, odd prefix
        dict(name="attn_verify", op="attn", kv="bf16", B=16, q_max=8, Hq=32, Hkv=8, d=128, prefix=16383, own_max=1000,
             lens=5),
        # d = 64, one query head per KV head, ragged
        dict(name="attn_d64", op="attn", kv="bf16", B=33, q_max=5, Hq=8, Hkv=8, d=64, prefix=4095, own_max=300, lens=6),
        # the largest: 256 requests on a 64K prefix
        dict(name="attn_large", op="attn", kv="bf16", B=256, q_max=1, Hq=32, Hkv=8, d=128, prefix=65536, own_max=2048,
             lens=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn"])
    if op != "attn":
        Hkv = rng.choice([1, 2, 4, 8])
        d, dv = rng.choice([(64, 64), (128, 128), (128, 128), (96, 96), (192, 128), (256, 256), (576, 0)])
        if dv == 0:
            Hkv = 1
        c = dict(op=op, n=_log_int(rng, 1, 32768), Hkv=Hkv, d=d, dv=dv, dtype=rng.choice(["bf16", "bf16", "fp32"]))
        if op == "write":
            c["padded"] = rng.random() < 0.5
        return c
    most = work(listed()[-1])
    while True:
        Hq, Hkv = rng.choice([(8, 8), (32, 8), (32, 8), (16, 2), (12, 4), (40, 8), (64, 8), (32, 1), (7, 1)])
        c = dict(op="attn", kv=rng.choice(["bf16", "e4m3"]), B=_log_int(rng, 1, 256),
                 q_max=rng.choice([1, 1, 1, 2, 4, 7, 16]), Hq=Hq, Hkv=Hkv, d=rng.choice([64, 128, 128]),
                 prefix=rng.choice([0, _log_int(rng, 1, 65536), _log_int(rng, 128, 65536), _log_int(rng, 128, 65536)]),
                 own_max=_log_int(rng, 1, 4096), lens=rng.randrange(1 << 20))
        w = work(c)
        N = sum(_lens(c)[0])
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and \
                N * c["Hq"] * c["prefix"] <= 1 << 29 and \
                N * (c["own_max"] + c["q_max"]) * c["Hkv"] * c["d"] <= 1 << 29:
            return c


def _lens(case):
    """Query tokens and own keys (the query tokens among them) of each request; a request without either is an empty slot
    of a padded batch.  From the case alone."""
    rng = random.Random(case["lens"])
    q, kv = [], []
    for b in range(case["B"]):
        ql = rng.randint(1, case["q_max"])
        q.append(ql)
        kv.append(0 if case["B"] > 4 and b % 31 == 30 else ql + rng.randint(0, case["own_max"] - 1))
    return q, kv


def _slots(case):
    """Positions of the padding rows of a padded write: every 16th row and the last."""
    return [i for i in range(case["n"]) if case["padded"] and (i % 16 == 15 or i == case["n"] - 1)]


def work(case):
    if case["op"] == "attn":
        ql, kl = _lens(case)
        N, Hq, Hkv, d, P = sum(ql), case["Hq"], case["Hkv"], case["d"], case["prefix"]
        row = Hkv * 2 * (2 * d if case["kv"] == "bf16" else d + 4)
        visible = sum(P + max(0, k - n + i + 1) for n, k in zip(ql, kl) for i in range(n))
        return {"bytes": (P + sum(kl)) * row + N * Hq * (4 * d + 4), "flops": 4 * d * Hq * visible}
    x = 2 if case["dtype"] == "bf16" else 4
    n, vectors = case["n"], case["Hkv"] * (2 if case["dv"] else 1)
    if case["op"] == "write":
        n -= len(_slots(case))
    per_row = case["Hkv"] * (case["d"] + case["dv"]) * (x + 1) + 4 * vectors
    return {"bytes": n * per_row + 4 * case["n"], "flops": 0}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _keys(g, shape, dtype=torch.bfloat16):
    """Keys as projections make them: a few channels much larger than the others."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.05
    return (x * torch.where(loud, 4.0, 0.8)).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "attn":
        ql, kl = _lens(case)
        N, Hq, Hkv, d, P = sum(ql), case["Hq"], case["Hkv"], case["d"], case["prefix"]
        cap = case["own_max"] + case["q_max"]  # rows kept for each request behind the prefix
        rows = P + case["B"] * cap
        s = dict(case=case, q=_normal(g, (N, Hq, d)), scale=d ** -0.5, cap=cap)
        k, v = _keys(g, (rows, Hkv, d)), _normal(g, (rows, Hkv, d))
        s["k_scale"] = s["v_scale"] = None
        if case["kv"] == "e4m3":
            (k, s["k_scale"]), (v, s["v_scale"]) = _quantize(k), _quantize(v)
        s["k"], s["v"] = k, v
        s["q_lens"] = torch.tensor(ql, device="cuda")
        s["own_lens"] = torch.tensor(kl, device="cuda")
        s["out"] = torch.empty((N, Hq, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((N, Hq), dtype=torch.float32, device="cuda")
        if own:
            import context_causal_attention_cp_gb300 as cpa

            # made once a decode step, used by every layer of the model
            s["plan"] = cpa.make_shared_plan(ql, kl, P, Hq, Hkv, own_row0=[P + b * cap for b in range(case["B"])])
            s["workspace"] = cpa.alloc_shared_workspace(s["plan"], d)
        return s
    n, Hkv, d, dv = case["n"], case["Hkv"], case["d"], case["dv"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "write":
        rows = n + n // 2 + 5
        s = dict(case=case, k=_keys(g, (n, Hkv, d), dtype), v=_normal(g, (n, Hkv, dv), dtype) if dv else None)
        slots = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32)
        pad = _slots(case)
        if pad:
            slots[torch.tensor(pad, device="cuda")] = -1
        s["slots"] = slots
    else:
        rows = -(-(n + n // 2 + 5) // PAGE) * PAGE
        pages = torch.randperm(rows // PAGE, generator=g, device="cuda")[:-(-n // PAGE)]
        idx = (pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)[:n]
        s = dict(case=case, idx=idx.to(torch.int32), out_k=torch.empty((n, Hkv, d), dtype=dtype, device="cuda"),
                 out_v=torch.empty((n, Hkv, dv), dtype=dtype, device="cuda") if dv else None)
    # what the cache holds before
    s["k_cache"], s["k_scale"] = _quantize(_keys(g, (rows, Hkv, d)))
    s["v_cache"], s["v_scale"] = _quantize(_normal(g, (rows, Hkv, dv))) if dv else (None, None)
    if own:
        import context_causal_attention_cp_gb300 as cpa

        s["cache"] = cpa.KVCache(s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"])
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


def _write(cache, scales, x, slots):
    codes, s = _quantize(x)
    kept = (slots >= 0).nonzero()[:, 0]
    at = slots[kept].long()
    cache.view(torch.uint8)[at] = codes.view(torch.uint8)[kept]
    scales[:, at] = s[:, kept]
    return cache, scales


def _values(codes, scales, rows):
    if scales is None:
        return codes[rows].float()
    return codes.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float() * scales[:, rows].t()[..., None]


def _attend(s):
    q, case, scale = s["q"].float(), s["case"], s["scale"]
    N, Hq, d = q.shape
    Hkv, P, cap = case["Hkv"], case["prefix"], s["cap"]
    g = Hq // Hkv
    req = torch.repeat_interleave(torch.arange(case["B"], device=q.device), s["q_lens"], output_size=N)
    first = torch.cumsum(s["q_lens"], 0) - s["q_lens"]
    seen = (s["own_lens"] - s["q_lens"])[req] + torch.arange(N, device=q.device) - first[req] + 1
    seen = torch.where(s["own_lens"][req] > 0, seen, 0)
    # the shared prefix: every query of the batch against the same keys
    pre = torch.arange(P, device=q.device)
    kp, vp = _values(s["k"], s["k_scale"], pre), _values(s["v"], s["v_scale"], pre)
    qh = q.view(N, Hkv, g, d).permute(1, 0, 2, 3).reshape(Hkv, N * g, d)
    sp = (qh @ kp.permute(1, 2, 0)).mul_(scale)
    # each request's own keys
    at = P + req[:, None] * cap + torch.arange(cap, device=q.device)
    hidden = torch.arange(cap, device=q.device) >= seen[:, None]
    ko, vo = _values(s["k"], s["k_scale"], at.reshape(-1)), _values(s["v"], s["v_scale"], at.reshape(-1))
    so = (q.view(N, Hkv, g, d) @ ko.view(N, cap, Hkv, d).permute(0, 2, 3, 1)).mul_(scale)
    so.masked_fill_(hidden[:, None, None, :], -math.inf)
    m = so.amax(-1)
    if P > 0:
        m = torch.maximum(m, sp.amax(-1).view(Hkv, N, g).permute(1, 0, 2))
    m = torch.where(m > -math.inf, m, 0.0)
    sp = sp.sub_(m.permute(1, 0, 2).reshape(Hkv, N * g, 1)).exp_()
    so = so.sub_(m[..., None]).exp_()
    total = so.sum(-1) + sp.sum(-1).view(Hkv, N, g).permute(1, 0, 2)
    o = so @ vo.view(N, cap, Hkv, d).permute(0, 2, 1, 3)
    o = o + (sp @ vp.permute(1, 0, 2)).view(Hkv, N, g, d).permute(1, 0, 2, 3)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return o.reshape(N, Hq, d).to(torch.bfloat16), (m + total.log()).reshape(N, Hq)


def run(s):
    case = s["case"]
    if case["op"] == "attn":
        if own:
            import context_causal_attention_cp_gb300 as cpa

            o, lse, _ = cpa.cp_attn_shared(s["plan"], s["q"], s["k"], s["v"], s["scale"], k_scale=s["k_scale"],
                                           v_scale=s["v_scale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
        else:
            o, lse = _attend(s)
        return {"o": o, "lse": lse}
    if case["op"] == "write":
        if own:
            import context_causal_attention_cp_gb300 as cpa

            cpa.cp_kv_quantize(s["cache"], s["k"], s["v"], s["slots"])
        else:
            _write(s["k_cache"], s["k_scale"], s["k"], s["slots"])
            if s["v"] is not None:
                _write(s["v_cache"], s["v_scale"], s["v"], s["slots"])
        return {"k": s["k_cache"], "k_scale": s["k_scale"], "v": s["v_cache"], "v_scale": s["v_scale"]}
    if own:
        import context_causal_attention_cp_gb300 as cpa

        k, v = cpa.cp_kv_dequantize(s["cache"], s["idx"], out_k=s["out_k"], out_v=s["out_v"])
    else:
        at, dtype = s["idx"].long(), s["out_k"].dtype
        k = _values(s["k_cache"], s["k_scale"], at).to(dtype)
        v = _values(s["v_cache"], s["v_scale"], at).to(dtype) if s["v_cache"] is not None else None
    return {"k": k, "v": v}


# ------------------------------------------------------------------------ exact --
def _exact_codes(x):
    """The definition in 64 bits: (code values [rows, Hkv, d], scales [Hkv, rows])."""
    x = x.double()
    a = torch.nan_to_num(x.abs(), nan=0.0, posinf=0.0).amax(-1)
    e = torch.ceil(torch.log2(a / 448.0))
    e = e + (a > 448.0 * torch.exp2(e)).double() - (a <= 448.0 * torch.exp2(e - 1)).double()
    e = torch.where(a > 0, e, -117.0).clamp(-117.0, 119.0)
    y = x / torch.exp2(e)[..., None]
    y = y.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.exp2(e).t()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        out = {}
        kept = s["slots"] >= 0
        at = s["slots"][kept].long()
        for name in ("k", "v"):
            if s[name] is None:
                out[name] = out[name + "_scale"] = None
                continue
            codes, scales = s[name + "_cache"].double(), s[name + "_scale"].double()
            new, sc = _exact_codes(s[name][kept])
            codes[at] = new
            scales[:, at] = sc
            out[name], out[name + "_scale"] = codes, scales
        return out
    if case["op"] == "read":
        out = {}
        for name in ("k", "v"):
            c = s[name + "_cache"]
            out[name] = None if c is None else \
                (c.double() * s[name + "_scale"].double().t()[:, :, None])[s["idx"].long()]
        return out
    ql, kl = _lens(case)
    Hq, Hkv, d, P = case["Hq"], case["Hkv"], case["d"], case["prefix"]
    g = Hq // Hkv

    def rows(name, lo, hi):
        x = s[name][lo:hi].double()
        return x if s[name + "_scale"] is None else x * s[name + "_scale"][:, lo:hi].double().t()[:, :, None]

    q = s["q"].double()
    kp, vp = rows("k", 0, P).transpose(0, 1), rows("v", 0, P).transpose(0, 1)  # [Hkv, P, d]
    os, ls, n0 = [], [], 0
    for b, (n, kv) in enumerate(zip(ql, kl)):
        lo = P + b * s["cap"]
        kb = torch.cat([kp, rows("k", lo, lo + kv).transpose(0, 1)], 1)
        vb = torch.cat([vp, rows("v", lo, lo + kv).transpose(0, 1)], 1)
        qb = q[n0:n0 + n].view(n, Hkv, g, d).permute(1, 2, 0, 3).reshape(Hkv, g * n, d)
        n0 += n
        x = (qb @ kb.transpose(1, 2)).view(Hkv, g, n, P + kv) * s["scale"]
        end = P + kv - n + 1 + torch.arange(n, device=q.device) if kv else torch.full((n,), P, device=q.device)
        x = x.masked_fill(torch.arange(P + kv, device=q.device)[None, :] >= end[:, None], -math.inf)
        lse = torch.logsumexp(x, -1) if P + kv else torch.full((Hkv, g, n), -math.inf, device=q.device).double()
        w = torch.exp(x - torch.where(lse > -math.inf, lse, 0.0)[..., None])
        o = (w.view(Hkv, g * n, P + kv) @ vb).view(Hkv, g, n, d)
        os.append(o.permute(2, 0, 1, 3).reshape(n, Hq, d))
        ls.append(lse.permute(2, 0, 1).reshape(n, Hq))
    return {"o": torch.cat(os), "lse": torch.cat(ls)}
