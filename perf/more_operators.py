"""Attention of many query rows over shared cached states, as cases to be measured.

Two operators over the paged K/V pools:

  cross   cross attention: every query token of a sequence attends all of an encoder's cached
          states (their number is another one than the queries'); single tokens, whole prompts
          in padded batches, and beams that share their encoder's states
  prefix  decode of a batch whose sequences share long prefixes, several groups of them: each
          prefix is attended once for all of its sequences, each sequence's own tokens beside it
          (causal among several query tokens), and the two are joined

own = False: each operator in elementary torch operations in fp32, rounded once at the end.
own = True: the calls a user makes of split_kv_decode_paged_gb300.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
_INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One token against a short clip's encoder states: the smallest call of every layer and step.
        dict(name="cross step 1", op="cross", R=1, beams=1, T=1, Hq=8, Hkv=8, D=64, page=16, q="f16", kv="f16", lo=375,
             hi=375, ragged=False, empty=False),
        # Beam search: 24 encoder rows, five beams each, one of the rows without states.
        dict(name="cross beams 24x5", op="cross", R=24, beams=5, T=1, Hq=16, Hkv=16, D=64, page=16, q="f16", kv="f16",
             lo=200, hi=1500, ragged=False, empty=True),
        # One token of each of 64 sequences over encoded documents (the heads and lengths of the GQA batch).
        dict(name="cross step 64", op="cross", R=64, beams=1, T=1, Hq=32, Hkv=8, D=128, page=16, q="bf16", kv="bf16",
             lo=512, hi=8192, ragged=False, empty=False),
        # A few tokens a sequence (drafts) over encoded documents in an E4M3 pool.
        dict(name="cross fp8 16x12", op="cross", R=16, beams=1, T=12, Hq=64, Hkv=8, D=128, page=128, q="bf16", kv="e4m3",
             lo=2048, hi=16384, ragged=False, empty=False),
        # Prompts of different lengths in a padded batch.
        dict(name="cross prompts 24x384", op="cross", R=24, beams=1, T=384, Hq=32, Hkv=8, D=128, page=16, q="bf16",
             kv="bf16", lo=100, hi=4096, ragged=True, empty=False),
        # The same work with one KV head a query head of 64 elements, 1500 states each.
        dict(name="cross heads 32x448", op="cross", R=32, beams=1, T=448, Hq=16, Hkv=16, D=64, page=16, q="f16", kv="f16",
             lo=1500, hi=1500, ragged=False, empty=False),
        # Long prompts over long documents: bound by arithmetic.
        dict(name="cross long 4x2048", op="cross", R=4, beams=1, T=2048, Hq=32, Hkv=8, D=128, page=64, q="bf16", kv="bf16",
             lo=8192, hi=8192, ragged=False, empty=False),
        # Four chats behind one short system prompt.
        dict(name="prefix 4", op="prefix", B=4, P=1, q_len=1, Hq=8, Hkv=2, D=64, page=16, q="f16", kv="f16", plo=500,
             phi=500, lo=1, hi=30, alone=0),
        # A batch behind one long system prompt that ends inside a page.
        dict(name="prefix 64", op="prefix", B=64, P=1, q_len=1, Hq=32, Hkv=8, D=128, page=16, q="bf16", kv="bf16",
             plo=8170, phi=8170, lo=64, hi=1024, alone=0),
        # Four draft tokens of each of 48 sequences behind three prompts, some sequences behind none.
        dict(name="prefix drafts 48x4", op="prefix", B=48, P=3, q_len=4, Hq=32, Hkv=8, D=128, page=64, q="f16", kv="f16",
             plo=1000, phi=12000, lo=4, hi=512, alone=5),
        # A mixed FP8 batch behind twelve prompts.
        dict(name="prefix fp8 256", op="prefix", B=256, P=12, q_len=1, Hq=64, Hkv=8, D=128, page=128, q="bf16", kv="e4m3",
             plo=300, phi=6000, lo=16, hi=2048, alone=10),
        # Many samples of one long document.
        dict(name="prefix 512", op="prefix", B=512, P=1, q_len=1, Hq=32, Hkv=8, D=128, page=64, q="bf16", kv="bf16",
             plo=32768, phi=32768, lo=128, hi=512, alone=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "prefix"])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 8, 12]) if Hkv < 16 else 1
    q = rng.choice(["f16", "bf16"])
    c = dict(op=op, Hq=G * Hkv, Hkv=Hkv, D=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128]), q=q,
             kv=rng.choice([q, q, "e4m3"]))
    if op == "cross":
        hi = _log_int(rng, 1, 20000)
        c.update(R=_log_int(rng, 1, 100), beams=rng.choice([1, 1, 2, 3, 5]), T=rng.choice([1, _log_int(rng, 2, 2048)]),
                 lo=max(1, int(hi * rng.uniform(0.05, 1))), hi=hi, ragged=rng.random() < 0.4, empty=rng.random() < 0.3)
        while not _fits(c):
            big = max(("T", "R", "hi"), key=lambda k: c[k] / {"T": 2048, "R": 100, "hi": 20000}[k])
            c[big] = max(1, c[big] * 2 // 3)
            c["lo"] = min(c["lo"], c["hi"])
        return c
    q_len = rng.choice([1, 1, 1, 2, 4, 5])
    P, phi, hi = _log_int(rng, 1, 16), _log_int(rng, 16, 40000), _log_int(rng, max(2, q_len), 3000)
    c.update(B=_log_int(rng, 2, 512), P=P, q_len=q_len, plo=max(1, int(phi * rng.uniform(0.05, 1))), phi=phi,
             lo=max(q_len, int(hi * rng.uniform(0.05, 1))), hi=hi, alone=rng.choice([0, 0, 1, 3]))
    while not _fits(c):
        big = max(("B", "phi", "hi"), key=lambda k: c[k] / {"B": 512, "phi": 40000, "hi": 3000}[k])
        c[big] = max(q_len, c[big] * 2 // 3)
        c["plo"], c["lo"] = min(c["plo"], c["phi"]), min(c["lo"], c["hi"])
    c["alone"] = min(c["alone"], c["B"] - 1)
    c["P"] = min(c["P"], c["B"] - c["alone"])
    return c


def _fits(c):
    w = work(c)
    return w["flops"] <= 1.0e12 and w["bytes"] <= 1.0e9


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread (both ends among them where n > 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _kv_lens(c):
    """Encoder lengths before the seed deals them out."""
    lens = _spread(c["R"], c["lo"], c["hi"])
    if c["empty"] and c["R"] > 1:
        lens[0] = 0
    return lens


def _q_lens(c):
    """Query tokens of every sequence (R * beams of them) before the seed deals them out."""
    n = c["R"] * c["beams"]
    return _spread(n, 1, c["T"]) if c["ragged"] else [c["T"]] * n


def _deal(lens, gen):
    return [lens[i] for i in torch.randperm(len(lens), generator=gen).tolist()]


def _members(c):
    """The prefix of every sequence before they are dealt out: even shares, -1 for those behind none."""
    return [-1] * c["alone"] + [i * c["P"] // (c["B"] - c["alone"]) for i in range(c["B"] - c["alone"])]


def work(c):
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    e = 1 if c["kv"] == "e4m3" else 2
    if c["op"] == "cross":
        kv, ql = _kv_lens(c), _q_lens(c)
        rows = sum(ql) * Hq
        # lengths and query counts are dealt apart: on average each query meets the mean length
        return {"bytes": sum(kv) * Hkv * D * 2 * e + rows * (4 * D + 4), "flops": 4.0 * rows * D * sum(kv) / len(kv)}
    pl, sl, of = _spread(c["P"], c["plo"], c["phi"]), _spread(c["B"], c["lo"], c["hi"]), _members(c)
    seen = sum(pl[i] for i in of if i >= 0) + sum(sl)
    rows = c["B"] * c["q_len"] * Hq
    return {"bytes": (sum(pl) + sum(sl)) * Hkv * D * 2 * e + rows * (4 * D + 4), "flops": 4.0 * c["q_len"] * Hq * D * seen}


# ----------------------------------------------------------------- inputs
def _table(page, lens, ids):
    """A block table that takes its pages from the list ids."""
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    return table


def _pool(c, pages, gen):
    """K or V pages of standard normal values; E4M3: codes, and a scale for each page and KV head."""
    shape = (pages, c["page"], c["Hkv"], c["D"])
    if c["kv"] != "e4m3":
        return torch.randn(shape, generator=gen, device="cuda", dtype=_DT[c["kv"]]), None
    x = torch.randn(shape, generator=gen, device="cuda")
    scale = x.abs().amax(dim=(1, 3)) / 448.0 * (1 + torch.rand((pages, c["Hkv"]), generator=gen, device="cuda"))
    return (x / scale[:, None, :, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device="cuda").manual_seed(seed + 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    act, page = _DT[c["q"]], c["page"]
    s = dict(c=c, act=act)
    groups = ([_deal(_kv_lens(c), host)] if c["op"] == "cross" else
              [_deal(_spread(c["P"], c["plo"], c["phi"]), host), _deal(_spread(c["B"], c["lo"], c["hi"]), host)])
    pages = 2 + sum(-(-n // page) for lens in groups for n in lens)
    ids = torch.randperm(pages, generator=host).tolist()
    tables = [_table(page, lens, ids).cuda() for lens in groups]
    s["k_pages"], s["k_scale"] = _pool(c, pages, dev)
    s["v_pages"], s["v_scale"] = _pool(c, pages, dev)
    if c["op"] == "cross":
        (s["kv_host"],), (s["table"],) = groups, tables
        s["kv_lens"] = torch.tensor(s["kv_host"], **i32)
        B, T = c["R"] * c["beams"], c["T"]
        lead = (B,) if T == 1 and not c["ragged"] else (B, T)
        s["q_lens"] = torch.tensor(_deal(_q_lens(c), host), **i32) if c["ragged"] else None
    else:
        (s["p_host"], s["kv_host"]), (s["p_table"], s["table"]) = groups, tables
        s["p_lens"], s["kv_lens"] = torch.tensor(s["p_host"], **i32), torch.tensor(s["kv_host"], **i32)
        s["prefix_of"] = _deal(_members(c), host)  # sequences of a group do not lie together
        lead = (c["B"],) if c["q_len"] == 1 else (c["B"], c["q_len"])
    # queries that pick some keys out of many: scores with a deviation of 2
    s["q"] = (2 * torch.randn((*lead, c["Hq"], c["D"]), generator=dev, device="cuda")).to(act)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:-1], dtype=torch.float32, device="cuda")
    if own:  # the plan and workspaces that a serving program keeps from step to step
        import split_kv_decode_paged_gb300 as fd
        if c["op"] == "cross":
            s["dec"] = fd.CrossDecoder.for_pools(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_host"],
                                                 beams=c["beams"])
        else:
            s["dec"] = fd.PrefixDecoder.for_pools(s["q"], s["k_pages"], s["v_pages"], s["p_table"], s["p_host"],
                                                  s["prefix_of"], s["table"], s["kv_host"])
    return s


# ------------------------------------------------------------ plain forms
def _gather(pool, scale, table, n):
    """Tokens [0, n) of block-table rows in fp32: [rows, Hkv, n, D]."""
    at = table.long().clamp(min=0)
    x = pool[at].float()
    if scale is not None:
        x = x * scale[at][:, :, None, :, None]
    return x.flatten(1, 2)[:, :n].transpose(1, 2)


def _soft(score):
    """Weights and log-sum-exp of masked scores (all masked: weights 0, -inf)."""
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m.masked_fill(m == -_INF, 0))
    total = p.sum(-1, keepdim=True)
    return p / total.masked_fill(total == 0, 1), (m + torch.log(total)).squeeze(-1)


def _run_cross(s):
    c = s["c"]
    R, n, T, Hkv, G, D = c["R"], c["beams"], c["T"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    q = s["q"].reshape(R, n * T, Hkv, G, D)
    out, lse = s["out"].view(q.shape), s["lse"].view(q.shape[:-1])
    for r, L in enumerate(s["kv_host"]):
        pages = -(-L // c["page"])
        k, v = (_gather(s[x + "_pages"], s[x + "_scale"], s["table"][r:r + 1, :max(1, pages)], L)[0] for x in "kv")
        rows = q[r].float().permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        if L:
            p, ls = _soft(rows @ k.transpose(1, 2) * D ** -0.5)
            o = p @ v
        else:
            o, ls = torch.zeros_like(rows), torch.full_like(rows[..., 0], -_INF)
        o, ls = o.view(Hkv, n * T, G, D).transpose(0, 1).to(s["act"]), ls.view(Hkv, n * T, G).transpose(0, 1)
        if s["q_lens"] is None:
            out[r], lse[r] = o, ls
        else:
            live = (torch.arange(T, device="cuda") < s["q_lens"][r * n:(r + 1) * n, None]).reshape(n * T, 1, 1)
            out[r], lse[r] = torch.where(live[..., None], o, out[r]), torch.where(live, ls, lse[r])
    return {"out": s["out"], "lse": s["lse"]}


def _run_prefix(s):
    c = s["c"]
    T, Hkv, G, D = c["q_len"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    q = s["q"].reshape(c["B"], T, Hkv, G, D)
    out, lse = s["out"].view(q.shape), s["lse"].view(q.shape[:-1])
    for g in range(-1, c["P"]):
        who = [b for b, p in enumerate(s["prefix_of"]) if p == g]
        if not who:
            continue
        longest = max(s["kv_host"][b] for b in who)
        b = torch.tensor(who, device="cuda")
        rows = q[b].float().permute(0, 2, 1, 3, 4)  # [n, Hkv, T, G, D]
        at = s["table"][b, :-(-longest // c["page"])]
        k, v = (_gather(s[x + "_pages"], s[x + "_scale"], at, longest) for x in "kv")
        seen = torch.arange(longest, device="cuda") < (s["kv_lens"][b][:, None] - T + 1 + torch.arange(T, device="cuda"))[..., None]
        score = (torch.einsum("nhtgd,nhkd->nhtgk", rows, k) * D ** -0.5).masked_fill(~seen[:, None, :, None], -_INF)
        if g >= 0:
            Lp = s["p_host"][g]
            kp, vp = (_gather(s[x + "_pages"], s[x + "_scale"], s["p_table"][g:g + 1, :-(-Lp // c["page"])], Lp)[0] for x in "kv")
            score = torch.cat([torch.einsum("nhtgd,hkd->nhtgk", rows, kp) * D ** -0.5, score], -1)
        p, ls = _soft(score)
        o = torch.einsum("nhtgk,nhkd->nhtgd", p[..., -longest:], v)
        if g >= 0:
            o = o + torch.einsum("nhtgk,hkd->nhtgd", p[..., :Lp], vp)
        out[b], lse[b] = o.transpose(1, 2).to(s["act"]), ls.transpose(1, 2)
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    c = s["c"]
    if not own:
        return _run_cross(s) if c["op"] == "cross" else _run_prefix(s)
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], lse=s["lse"])
    if c["op"] == "cross":
        s["dec"](s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], q_lens=s["q_lens"], **scales)
    else:
        s["dec"](s["q"], s["k_pages"], s["v_pages"], s["p_table"], s["p_lens"], s["table"], s["kv_lens"], **scales)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """One sequence and query token at a time (a block of them for a prompt), from the formulas."""
    c, s = dict(case), prepare(case, seed)
    page, Hq, Hkv, D = c["page"], c["Hq"], c["Hkv"], c["D"]
    out, lse = s["out"].double(), s["lse"].double()

    def states(x, row, n):
        """Tokens [0, n) of a block-table row in 64 bits: [n, Hkv, D]."""
        ids = row[:-(-n // page)].long()
        y = s[x + "_pages"][ids].double()
        if s[x + "_scale"] is not None:
            y *= s[x + "_scale"][ids].double()[:, None, :, None]
        return y.reshape(-1, Hkv, D)[:n]

    def attend(q, k, v):
        """q [m, Hq, D] over all of k and v [n, Hkv, D]."""
        m, n = q.shape[0], k.shape[0]
        if n == 0:
            return torch.zeros_like(q), torch.full((m, Hq), -_INF, dtype=torch.float64, device="cuda")
        o, l = torch.empty_like(q), torch.empty((m, Hq), dtype=torch.float64, device="cuda")
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            z = q[:, h] @ k[:, kv].T / math.sqrt(D)
            l[:, h] = torch.logsumexp(z, -1)
            o[:, h] = torch.exp(z - l[:, h, None]) @ v[:, kv]
        return o, l

    q = s["q"].double()
    if c["op"] == "cross":
        T = 1 if q.dim() == 3 else q.shape[1]
        q, o4, l3 = q.view(-1, T, Hq, D), out.view(-1, T, Hq, D), lse.view(-1, T, Hq)
        counts = [T] * q.shape[0] if s["q_lens"] is None else s["q_lens"].tolist()
        for r, L in enumerate(s["kv_host"]):
            k, v = states("k", s["table"][r], L), states("v", s["table"][r], L)
            for b in range(r * c["beams"], (r + 1) * c["beams"]):
                o4[b, :counts[b]], l3[b, :counts[b]] = attend(q[b, :counts[b]], k, v)
        return {"out": out, "lse": lse}
    T = c["q_len"]
    q, o4, l3 = q.view(-1, T, Hq, D), out.view(-1, T, Hq, D), lse.view(-1, T, Hq)
    for g in range(-1, c["P"]):
        before = {x: states(x, s["p_table"][g], s["p_host"][g]) for x in "kv"} if g >= 0 else None
        for b in (i for i, p in enumerate(s["prefix_of"]) if p == g):
            k, v = (states(x, s["table"][b], s["kv_host"][b]) for x in "kv")
            if before is not None:
                k, v = torch.cat([before["k"], k]), torch.cat([before["v"], v])
            for t in range(T):
                n = k.shape[0] - T + 1 + t
                o4[b, t:t + 1], l3[b, t:t + 1] = attend(q[b, t:t + 1], k[:n], v[:n])
    return {"out": out, "lse": lse}
