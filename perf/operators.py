"""The cache-management operators of the paged decode path, as cases to be measured.

Four operators of one serving step over a paged K/V cache:

  append   RMS norm of every query and key head, rotary embedding and the write of K and V
           into the paged pools, for one or many new tokens per sequence
  weights  the decode step that also adds every cached token's attention weight (summed over
           the query heads of its KV head) to a running total
  evict    the cached tokens with the smallest totals leave a sequence that passed its budget,
           the others move up in order
  diff     differential attention over the paged cache: softmax map 1 minus lambda times
           softmax map 2, then the per-head norm

own = False: each operator in elementary torch operations in fp32, rounded once at the end.
own = True: the calls a user makes of split_kv_decode_paged_gb300.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One sequence takes one token: the smallest call of a chat's every step (32 query, 8 KV heads).
        dict(name="append 1x1", op="append", B=1, T=1, Hq=32, Hkv=8, D=128, page=64, kv="bf16", rd=128,
             interleaved=False, ragged=False, ctx=4096),
        # A serving batch takes one token each into an E4M3 cache (the shape of the mixed FP8 batch).
        dict(name="append fp8 256x1", op="append", B=256, T=1, Hq=64, Hkv=8, D=128, page=128, kv="e4m3", rd=128,
             interleaved=False, ragged=False, ctx=32768),
        # Prompts of different lengths in one padded batch (prefill), 16-token pages.
        dict(name="append prompts 8x4096", op="append", B=8, T=4096, Hq=32, Hkv=8, D=128, page=16, kv="bf16", rd=128,
             interleaved=False, ragged=True, ctx=0),
        # Four MHA heads over 256 tokens: a call of a few microseconds.
        dict(name="weights tiny", op="weights", B=1, Hq=4, Hkv=4, D=64, page=16, kv="f16", lo=256, hi=256, q_len=1,
             empty=False),
        # The GQA batch: 64 sequences of 512 to 8192 tokens.
        dict(name="weights batch 64", op="weights", B=64, Hq=32, Hkv=8, D=128, page=16, kv="bf16", lo=512, hi=8192,
             q_len=1, empty=False),
        # One long document, split over the SMs.
        dict(name="weights long 131072", op="weights", B=1, Hq=32, Hkv=8, D=128, page=64, kv="bf16", lo=131072,
             hi=131072, q_len=1, empty=False),
        # One sequence 256 tokens past its budget.
        dict(name="evict 1x2304", op="evict", B=1, Hkv=8, D=128, page=16, kv="bf16", lo=2304, hi=2304, budget=2048,
             sinks=4, recent=256),
        # A batch whose longer half is past its budget.
        dict(name="evict batch 64", op="evict", B=64, Hkv=8, D=128, page=16, kv="bf16", lo=512, hi=8192, budget=4096,
             sinks=4, recent=1024),
        # Long documents of an E4M3 cache halved, codes moved between pages of different scales.
        dict(name="evict fp8 4x65536", op="evict", B=4, Hkv=8, D=128, page=128, kv="e4m3", lo=60000, hi=65536,
             budget=32768, sinks=16, recent=4096),
        # One sequence of 512 tokens, four heads of two 64-wide maps.
        dict(name="diff tiny", op="diff", B=1, Hq=4, Hkv=4, D=128, page=16, kv="f16", lo=512, hi=512, q_len=1, norm=True,
             empty=False),
        # A batch of 64 with grouped heads.
        dict(name="diff batch 64", op="diff", B=64, Hq=32, Hkv=8, D=128, page=16, kv="bf16", lo=512, hi=8192, q_len=1,
             norm=True, empty=False),
        # Four draft tokens per sequence verified over an E4M3 cache, causal among them.
        dict(name="diff fp8 4 tokens", op="diff", B=8, Hq=32, Hkv=8, D=128, page=64, kv="e4m3", lo=8192, hi=32768,
             q_len=4, norm=True, empty=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "weights", "evict", "diff"])
    kv = rng.choice(["f16", "bf16", "e4m3"])
    page = rng.choice([16, 32, 48, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 12])
    if op == "append":
        D = rng.choice([64, 128])
        tokens = _log_int(rng, 1, 20000)
        T = min(4096, _log_int(rng, 1, tokens))
        return dict(op=op, B=max(1, tokens // T), T=T, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, kv=kv,
                    rd=rng.choice([D, D // 2, D // 4 + 2]), interleaved=rng.random() < 0.4, ragged=rng.random() < 0.5,
                    ctx=_log_int(rng, 1, 30000))
    if op == "evict":
        hi = _log_int(rng, 2, 65536)
        B = max(1, min(128, _log_int(rng, 1, max(2, 2000000 // (hi * Hkv)))))
        budget = max(1, int(hi * rng.uniform(0.3, 0.98)))
        sinks = min(budget, rng.choice([0, 1, 4, 16]))
        return dict(op=op, B=B, Hkv=Hkv, D=rng.choice([64, 128]), page=page, kv=kv, lo=max(1, int(hi * rng.uniform(0.2, 1))),
                    hi=hi, budget=budget, sinks=sinks, recent=min(budget - sinks, int(budget * rng.uniform(0, 0.6))))
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    hi = _log_int(rng, 8, 100000)
    B = max(1, min(200, _log_int(rng, 1, max(2, 2500000 // (hi * Hkv)))))
    c = dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=rng.choice([64, 128]), page=page, kv=kv,
             lo=max(q_len, int(hi * rng.uniform(0.05, 1))), hi=hi, q_len=q_len, empty=q_len == 1 and B > 1 and rng.random() < 0.5)
    return dict(c, norm=rng.random() < 0.7) if op == "diff" else c


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread (both ends among them where n > 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(c):
    """The case's lengths before the seed deals them to the sequences."""
    if c["op"] == "append":
        return _spread(c["B"], max(1, c["T"] // 64), c["T"]) if c["ragged"] else [c["T"]] * c["B"]
    lens = _spread(c["B"], c["lo"], c["hi"])
    if c.get("empty"):
        lens[0] = 0
    return lens


def _width(c):
    return 1 if c["kv"] == "e4m3" else 2


def work(c):
    lens, e, D, Hkv = _lens(c), _width(c), c["D"], c["Hkv"]
    if c["op"] == "append":
        n, Hq = sum(lens), c["Hq"]
        # q in and out, k and v in at 16 bits, k and v out in the cache's type, a row of cosines and sines
        # for every distinct position (the longest run's, and up to one for every other token)
        rows = min(n, c["ctx"] + c["T"])
        return {"bytes": n * D * (2 * Hq * 2 + 2 * Hkv * 2 + 2 * Hkv * e) + rows * c["rd"] * 4 + 4 * n,
                "flops": n * D * (Hq + Hkv) * 8}
    tok = sum(lens)
    if c["op"] == "evict":
        n = sum(min(L, c["budget"]) for L in lens)
        # every total read, the kept ones and their indices written, the kept rows of K and V read and written
        return {"bytes": Hkv * (4 * tok + 8 * n + 4 * n * D * e), "flops": Hkv * tok}
    rows = c["B"] * c["q_len"] * c["Hq"]
    kv = tok * Hkv * D * 2 * e
    if c["op"] == "weights":
        # K and V once, the totals read and written, q, out and lse
        return {"bytes": kv + 8 * tok * Hkv + rows * (4 * D + 4),
                "flops": 4.0 * tok * c["q_len"] * c["Hq"] * D}
    # two maps over half of K's width each and the whole of V's: 2 D + 4 D operations a token and head
    return {"bytes": kv + rows * (4 * D + 8), "flops": 6.0 * tok * c["q_len"] * c["Hq"] * D}


# ----------------------------------------------------------------- inputs
def _pages(c, lens, extra, gen):
    """A block table over randomly dealt pages for the lengths, and the pool's pages (extra: spare ones)."""
    need = [-(-n // c["page"]) for n in lens]
    total = sum(need) + extra
    perm = torch.randperm(total, generator=gen)
    table, at = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    return table, total, perm[at:]


def _pool(c, pages, dev):
    """K or V pages of standard normal values; E4M3: codes, and a scale for each page and KV head."""
    shape = (pages, c["page"], c["Hkv"], c["D"])
    x = torch.randn(shape, generator=dev, device="cuda", dtype=torch.float32 if c["kv"] == "e4m3" else _DT[c["kv"]])
    if c["kv"] != "e4m3":
        return x, None
    scale = x.abs().amax(dim=(1, 3)) / 448.0 * (1 + torch.rand((pages, c["Hkv"]), generator=dev, device="cuda"))
    return (x / scale[:, None, :, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device="cuda").manual_seed(seed + 1)
    order = torch.randperm(c["B"], generator=host).tolist()
    lens = [_lens(c)[i] for i in order]
    act = torch.float16 if c["kv"] == "f16" else torch.bfloat16  # type of q, out and new tokens
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(c=c, act=act)
    normal = lambda *shape: torch.randn(shape, generator=dev, device="cuda")  # noqa: E731

    if c["op"] == "append":
        B, T, D = c["B"], c["T"], c["D"]
        ctx = [_spread(B, 0, c["ctx"])[::-1][i] if B > 1 else c["ctx"] for i in order]
        table, pages, _ = _pages(c, [a + n for a, n in zip(ctx, lens)], 2, host)
        s["k_pages"], s["k_scale"] = _pool(c, pages, dev)
        s["v_pages"], s["v_scale"] = _pool(c, pages, dev)
        qkv = normal(B, T, (c["Hq"] + 2 * c["Hkv"]) * D).to(act)  # the output of the fused projection
        q, k, v = qkv.split([c["Hq"] * D, c["Hkv"] * D, c["Hkv"] * D], dim=-1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (c["Hq"], D)), k.unflatten(-1, (c["Hkv"], D)), v.unflatten(-1, (c["Hkv"], D))
        s["q_out"] = torch.zeros(B, T, c["Hq"], D, dtype=act, device="cuda")
        s["qw"], s["kw"] = (1 + 0.2 * normal(D)).to(act), (1 + 0.2 * normal(D)).to(act)
        # positions run on from every token a sequence ever had: evicted ones still count
        gone = torch.randint(0, 1000, (B,), generator=host)
        s["pos"] = (torch.tensor(ctx) + gone).to(**i32)
        angle = torch.arange(c["ctx"] + T + 1000, dtype=torch.float64, device="cuda")[:, None] * (
            10000.0 ** (-torch.arange(c["rd"] // 2, dtype=torch.float64, device="cuda") / (c["rd"] // 2)))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["table"], s["lens"] = table.cuda(), torch.tensor(ctx, **i32)
        s["new"] = torch.tensor(lens, **i32) if c["ragged"] else None
        return s

    table, pages, spare = _pages(c, lens, sum(-(-min(n, c["budget"]) // c["page"]) for n in lens) if c["op"] == "evict" else 2, host)
    s["k_pages"], s["k_scale"] = _pool(c, pages, dev)
    s["v_pages"], s["v_scale"] = _pool(c, pages, dev)
    s["table"], s["lens"] = table.cuda(), torch.tensor(lens, **i32)
    room = table.shape[1] * c["page"]
    if c["op"] != "diff":
        # totals of earlier steps: a few tokens hold most of the weight, some none at all
        w = torch.rand((c["B"], c["Hkv"], room), generator=dev, device="cuda")
        s["w"] = 20 * w.square().square() * (torch.rand(w.shape, generator=dev, device="cuda") > 0.03)
        s["w_out"] = torch.zeros_like(s["w"])
    if c["op"] == "evict":
        # the kept rows go to fresh pages, as where others still hold the old ones
        new, at = torch.full((c["B"], table.shape[1]), -1, dtype=torch.int32), 0
        for b, n in enumerate(lens):
            m = -(-min(n, c["budget"]) // c["page"])
            new[b, :m] = spare[at:at + m].to(torch.int32)
            at += m
        s["new_table"] = new.cuda()
        return s
    lead = (c["B"],) if c["q_len"] == 1 else (c["B"], c["q_len"])
    s["q"] = normal(*lead, c["Hq"], c["D"]).to(act)
    if c["op"] == "diff":
        s["lam"] = 0.2 + 0.6 * torch.rand(c["Hq"], generator=dev, device="cuda")
        s["nw"] = (1 + 0.2 * normal(c["D"])).to(act) if c["norm"] else None
    if own:  # the plan and workspaces that a serving program keeps from step to step
        import split_kv_decode_paged_gb300 as fd
        if c["op"] == "diff":
            s["dec"] = fd.DiffDecoder.for_pools(s["q"], s["k_pages"], s["v_pages"], s["table"], lens)
        else:
            s["dec"] = fd.PagedDecoder.for_pools(s["q"], s["k_pages"], s["v_pages"], s["table"], lens, track_weights=True)
    return s


# ------------------------------------------------------------ plain forms
def _rms(x, w, eps):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _rotate(x, cos, sin, interleaved):
    """x [n, H, D], cos and sin [n, rd / 2]."""
    rd = 2 * cos.shape[-1]
    cos, sin, r, rest = cos[:, None], sin[:, None], x[..., :rd], x[..., rd:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rd // 2], r[..., rd // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([r, rest], -1)


def _store(pool, page, slot, x, scale):
    """Rows x [n, H, D] into their pages, rounded once."""
    if scale is None:
        pool[page, slot] = x.to(pool.dtype)
    else:
        codes = (x / scale[page][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        pool.view(torch.uint8)[page, slot] = codes.view(torch.uint8)


def _run_append(s):
    c = s["c"]
    t = torch.arange(c["T"], device="cuda")
    live = (t[None] < s["new"][:, None] if s["new"] is not None else torch.ones(c["B"], c["T"], dtype=torch.bool, device="cuda"))
    b, i = live.nonzero(as_tuple=True)
    at = s["lens"].long()[b] + i
    page, slot = s["table"].long()[b, at // c["page"]], at % c["page"]
    pos = s["pos"].long()[b] + i
    cos, sin = s["cos"][pos], s["sin"][pos]
    s["q_out"][b, i] = _rotate(_rms(s["q"][b, i], s["qw"], 1e-6), cos, sin, c["interleaved"]).to(s["act"])
    _store(s["k_pages"], page, slot, _rotate(_rms(s["k"][b, i], s["kw"], 1e-6), cos, sin, c["interleaved"]), s["k_scale"])
    _store(s["v_pages"], page, slot, s["v"][b, i].float(), s["v_scale"])
    return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}


def _gather(pool, scale, table):
    """The pages of every sequence in fp32: [B, Hkv, tokens, D]."""
    at = table.long().clamp(min=0)
    x = pool[at].float()
    if scale is not None:
        x = x * scale[at][:, :, None, :, None]
    return x.flatten(1, 2).transpose(1, 2)


def _softmax(score, seen):
    """Weights and log-sum-exp over the seen tokens (none seen: weights 0, -inf)."""
    score = score.masked_fill(~seen, -_INF)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - m.masked_fill(m == -_INF, 0))
    total = p.sum(-1, keepdim=True)
    return p / total.masked_fill(total == 0, 1), (m + torch.log(total)).squeeze(-1)


def _seen(s, n):
    """[B, 1, q_len, 1, n]: the tokens that each query token sees."""
    c = s["c"]
    end = s["lens"].long()[:, None] - c["q_len"] + 1 + torch.arange(c["q_len"], device="cuda")
    return (torch.arange(n, device="cuda") < end[:, :, None])[:, None, :, None]


def _attend(s, q, k, v):
    """q [B, q_len, Hkv, G, d] over k [B, Hkv, n, d] and v: outputs, lse and weights, heads behind query tokens."""
    score = torch.einsum("bqhgd,bhnd->bhqgn", q.float(), k) * q.shape[-1] ** -0.5
    p, lse = _softmax(score, _seen(s, k.shape[2]))
    return torch.einsum("bhqgn,bhnd->bqhgd", p, v), lse.transpose(1, 2), p


def _run_weights(s):
    c = s["c"]
    k, v = _gather(s["k_pages"], s["k_scale"], s["table"]), _gather(s["v_pages"], s["v_scale"], s["table"])
    q = s["q"].reshape(c["B"], c["q_len"], c["Hkv"], -1, c["D"])
    out, lse, p = _attend(s, q, k, v)
    live = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None, None]
    total = torch.where(live, s["w"] + p.sum((2, 3)), s["w_out"])
    return {"out": out.reshape(s["q"].shape).to(s["act"]), "lse": lse.reshape(s["q"].shape[:-1]), "weights": total}


def _run_diff(s):
    c, d = s["c"], s["c"]["D"] // 2
    k, v = _gather(s["k_pages"], s["k_scale"], s["table"]), _gather(s["v_pages"], s["v_scale"], s["table"])
    q = s["q"].reshape(c["B"], c["q_len"], c["Hkv"], -1, c["D"])
    o1, l1, _ = _attend(s, q[..., :d], k[..., :d], v)
    o2, l2, _ = _attend(s, q[..., d:], k[..., d:], v)
    o = o1 - s["lam"].reshape(c["Hkv"], -1, 1) * o2
    if s["nw"] is not None:
        o = _rms(o, s["nw"], 1e-5) * 0.2
    return {"out": o.reshape(s["q"].shape).to(s["act"]), "lse": torch.stack([l1, l2], -1).reshape(*s["q"].shape[:-1], 2)}


def _run_evict(s):
    c, L = s["c"], s["lens"].long()
    B, H, room = s["w"].shape
    budget, t = c["budget"], torch.arange(room, device="cuda")
    n = L.clamp(max=budget)
    # what stays whatever its total: the first tokens, the last ones, all of a short sequence
    stays = (t < c["sinks"]) | (t >= (L - c["recent"])[:, None]) | (L <= budget)[:, None]
    rank = torch.where(stays[:, None], _INF, s["w"]).masked_fill((t >= L[:, None])[:, None], -_INF)
    best = rank.sort(dim=-1, descending=True, stable=True).indices
    chosen = torch.zeros(B, H, room, dtype=torch.bool, device="cuda").scatter_(-1, best, (t < n[:, None])[:, None].expand(B, H, room))
    b, h, src = chosen.nonzero(as_tuple=True)  # in order of their places
    at = (chosen.cumsum(-1) - 1)[b, h, src]
    kept = torch.full((B, H, budget), -1, dtype=torch.int32, device="cuda")
    kept[b, h, at] = src.int()
    total = s["w_out"].masked_fill((t < L[:, None])[:, None], 0)
    total[b, h, at] = s["w"][b, h, src]
    old, slot = s["table"].long()[b, src // c["page"]], src % c["page"]
    new, to = s["new_table"].long()[b, at // c["page"]], at % c["page"]
    for pool, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])):
        if scale is None:
            pool[new, to, h] = pool[old, slot, h]
        else:
            x = pool.view(torch.uint8)[old, slot, h].view(torch.float8_e4m3fn).float() * scale[old, h][:, None] / scale[new, h][:, None]
            pool.view(torch.uint8)[new, to, h] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return {"k": s["k_pages"], "v": s["v_pages"], "weights": total, "lens": n.int(), "kept": kept}


def run(s):
    c = s["c"]
    if not own:
        return {"append": _run_append, "weights": _run_weights, "evict": _run_evict, "diff": _run_diff}[c["op"]](s)
    import split_kv_decode_paged_gb300 as fd
    pools = (s["k_pages"], s["v_pages"], s["table"], s["lens"])
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "append":
        fd.append_kv_norm(s["q"], s["k"], s["v"], *pools, q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, rotary_cos=s["cos"],
                          rotary_sin=s["sin"], interleaved=c["interleaved"], positions=s["pos"], new_lens=s["new"],
                          q_out=s["q_out"], **scales)
        return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}
    if c["op"] == "weights":
        out, lse, total = s["dec"].decode_weights(s["q"], *pools, s["w"], weights_out=s["w_out"], **scales)
        return {"out": out, "lse": lse, "weights": total}
    if c["op"] == "diff":
        out, lse = s["dec"](s["q"], *pools, s["lam"], norm_weight=s["nw"], eps=1e-5, out_scale=0.2 if c["norm"] else 1.0, **scales)
        return {"out": out, "lse": lse}
    n, kept = fd.evict_kv(*pools, s["w"], c["budget"], sinks=c["sinks"], recent=c["recent"], dst_table=s["new_table"],
                          weights_out=s["w_out"], **scales)
    return {"k": s["k_pages"], "v": s["v_pages"], "weights": s["w_out"], "lens": n, "kept": kept}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """One sequence (and for a moved or appended row, one token range) at a time, from the formulas."""
    c, s = dict(case), prepare(case, seed)
    page, lens, table = c["page"], s["lens"].tolist(), s["table"].tolist()

    def tokens(pool, scale, row, n, units=False):
        """Tokens [0, n) of a block-table row: [n, Hkv, D]."""
        ids = torch.tensor(row[:-(-n // page)], dtype=torch.long, device="cuda")
        x = pool[ids].double()
        if scale is not None:
            x *= scale[ids].double()[:, None, :, None]
        return x.reshape(-1, c["Hkv"], c["D"])[:n]

    def place(at, row):
        """Page and slot of the token places `at` (a tensor) of a block-table row."""
        return torch.tensor(row, dtype=torch.long, device="cuda")[at // page], at % page

    if c["op"] == "append":
        q_out, kp, vp = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
        news = s["new"].tolist() if s["new"] is not None else [c["T"]] * c["B"]
        rd = c["rd"]
        first = torch.arange(rd // 2, device="cuda") * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else rd // 2)

        def turned(x, w, cos, sin):
            y = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
            z = y.clone()
            z[..., first] = y[..., first] * cos - y[..., second] * sin
            z[..., second] = y[..., first] * sin + y[..., second] * cos
            return z

        for b in range(c["B"]):
            n, p0 = news[b], int(s["pos"][b])
            cos, sin = (s[x][p0:p0 + n].double()[:, None] for x in ("cos", "sin"))
            q_out[b, :n] = turned(s["q"][b, :n].double(), s["qw"], cos, sin)
            pg, sl = place(torch.arange(lens[b], lens[b] + n, device="cuda"), table[b])
            k, v = turned(s["k"][b, :n].double(), s["kw"], cos, sin), s["v"][b, :n].double()
            if s["k_scale"] is not None:
                k = (k / s["k_scale"][pg].double()[..., None]).clamp(-448, 448)
                v = (v / s["v_scale"][pg].double()[..., None]).clamp(-448, 448)
            kp[pg, sl], vp[pg, sl] = k, v
        return {"q": q_out, "k": kp, "v": vp}

    if c["op"] == "evict":
        kp, vp, total = s["k_pages"].double(), s["v_pages"].double(), s["w_out"].double()
        budget = c["budget"]
        kept = torch.full((c["B"], c["Hkv"], budget), -1, dtype=torch.int32)
        new_table = s["new_table"].tolist()
        for b, L in enumerate(lens):
            total[b, :, :L] = 0
            for h in range(c["Hkv"]):
                w = s["w"][b, h, :L].double()
                keep = torch.arange(L, device="cuda")
                if L > budget:
                    mid = keep[c["sinks"]:L - c["recent"]]
                    many = budget - c["sinks"] - c["recent"]
                    low_first = torch.sort(-w[mid], stable=True).indices[:many]
                    keep = torch.cat([keep[:c["sinks"]], mid[low_first].sort().values, keep[L - c["recent"]:]])
                n = keep.numel()
                kept[b, h, :n] = keep.int().cpu()
                total[b, h, :n] = w[keep]
                op, osl = place(keep, table[b])
                np_, nsl = place(torch.arange(n, device="cuda"), new_table[b])
                for out, pool, scale in ((kp, s["k_pages"], s["k_scale"]), (vp, s["v_pages"], s["v_scale"])):
                    if scale is None:
                        out[np_, nsl, h] = pool[op, osl, h].double()
                    else:
                        code = pool.view(torch.uint8)[op, osl, h].view(torch.float8_e4m3fn).double()
                        ratio = scale[op, h].double() / scale[np_, h].double()
                        out[np_, nsl, h] = (code * ratio[:, None]).clamp(-448, 448)
        return {"k": kp, "v": vp, "weights": total, "lens": torch.tensor([min(L, budget) for L in lens], dtype=torch.int32),
                "kept": kept}

    B, T, Hq, Hkv, D = c["B"], c["q_len"], c["Hq"], c["Hkv"], c["D"]
    q = s["q"].double().reshape(B, T, Hkv, Hq // Hkv, D)
    out = torch.zeros(B, T, Hkv, Hq // Hkv, D, dtype=torch.float64, device="cuda")
    maps = 1 if c["op"] == "weights" else 2
    lse = torch.full((B, T, Hkv, Hq // Hkv, maps), -_INF, dtype=torch.float64, device="cuda")
    total = s["w_out"].double() if maps == 1 else None
    w = D // maps
    for b, L in enumerate(lens):
        if L == 0:
            continue
        k, v = (tokens(s[x + "_pages"], s[x + "_scale"], table[b], L) for x in "kv")
        if maps == 1:
            total[b, :, :L] = s["w"][b, :, :L].double()
        for i in range(T):
            n = L - T + i + 1
            for m in range(maps):
                z = torch.einsum("hgd,nhd->hgn", q[b, i, ..., m * w:(m + 1) * w], k[:n, :, m * w:(m + 1) * w]) / math.sqrt(w)
                lse[b, i, ..., m] = torch.logsumexp(z, -1)
                p = torch.exp(z - lse[b, i, ..., m, None])
                o = torch.einsum("hgn,nhd->hgd", p, v[:n])
                out[b, i] += o if m == 0 else -s["lam"].double().reshape(Hkv, -1, 1) * o
                if maps == 1:
                    total[b, :, :n] += p.sum(1)
    if c["op"] == "weights":
        return {"out": out.reshape(s["q"].shape), "lse": lse.reshape(s["q"].shape[:-1]), "weights": total}
    if s["nw"] is not None:
        out = out / (out.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * s["nw"].double() * 0.2
    return {"out": out.reshape(s["q"].shape), "lse": lse.reshape(*s["q"].shape[:-1], 2)}
