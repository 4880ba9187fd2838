"""Plain float64 definitions of cross attention and of decode behind shared
prefixes on CPU tensors, with the error bounds the tests hold the kernels to,
and the seeded cases they run on.

Unused slots and pages hold NaN (E4M3: NaN codes and NaN scales of unused
pages): what is read of them shows.

Bounds.  A score's error (attend in cache_ref): e_s.  A weight exp(s - m) is
then off by e_s relative (both s and m: 2 e_s), by the exponential's own few
2^-22, and by its rounding r_p for the product with V: half a step of the
product's type (bf16 2^-8, f16 2^-11).  E4M3 pools: f16, or where the scales of a
chunk's pages differ by more than 8 bf16, under f16 queries pairs of bf16 (2^-16).
f16 weights below 2^-14 are off by up to 2^-25 instead, relative to a unit of at
most twice the largest |v| can be: n 2^-24 max |v| in all.  The sums over n tokens
in fp32 add at most n 2^-24 each, in numerator and denominator.  Together
    sum p |v| (r_p + 4 e_s + n 2^-23 + 2^-18) + n 2^-24 max |v|
and then the output's own rounding.  The log-sum-exp: 2 e_s + n 2^-24 + 2^-18
(1 + |lse|).  Decode behind prefixes joins a second pass over the own tokens,
whose weights are f16 but for bf16 pools (pairs of bf16): r_p at least 2^-11.
"""
import torch

from tests.cache_ref import HALF_STEP, make_table, rounding, seq_tokens, values

NAN = float("nan")


def r_p(q_dtype, kv_dtype, wide=False):
    if kv_dtype == torch.float8_e4m3fn:
        return 2.0 ** -8 if wide and q_dtype == torch.bfloat16 else 2.0 ** -11
    return HALF_STEP[kv_dtype]


def pools(gen, lens_tables, pages, ps, H, D, kv, wide=False):
    """K and V pools (and scales) with NaN wherever no table's live slot lies;
    wide: E4M3 scales of very different sizes."""
    live = torch.zeros(pages, ps, dtype=torch.bool)
    for lens, table in lens_tables:
        for b, L in enumerate(lens):
            for j in range(-(-int(L) // ps)):
                live[int(table[b, j]), :min(ps, int(L) - j * ps)] = True
    out = []
    for _ in "kv":
        x = torch.randn((pages, ps, H, D), generator=gen)
        if kv != torch.float8_e4m3fn:
            x[~live] = NAN
            out += [x.to(kv), None]
            continue
        scale = x.abs().amax(dim=(1, 3)) / 448.0 * (1 + torch.rand((pages, H), generator=gen))
        codes = (x / scale[:, None, :, None]).to(kv)
        if wide:
            scale = scale * torch.exp2(torch.randint(-6, 7, scale.shape, generator=gen).float())
        codes.view(torch.uint8)[~live] = 0x7f
        scale[~live.any(dim=1)] = NAN
        out += [codes, scale]
    return out


def attend_many(q, k, v, n_seen=None):
    """q [m, Hq, D] over k and v [n, Hkv, D] in float64: out [m, Hq, D],
    sum p |v|, lse [m, Hq] and the scores' error bound; row i sees the first
    n_seen[i] tokens (all of them)."""
    m, Hq, D = q.shape
    n, Hkv = k.shape[:2]
    qq = q.reshape(m, Hkv, Hq // Hkv, D)
    if n == 0:
        z = torch.zeros(m, Hq, D, dtype=torch.float64)
        return z, z, torch.full((m, Hq), -float("inf"), dtype=torch.float64), 0.0
    s = torch.einsum("mhgd,nhd->mhgn", qq, k) * D ** -0.5
    mag = torch.einsum("mhgd,nhd->mhgn", qq.abs(), k.abs()) * D ** -0.5
    err = float(mag.max()) * (2.0 ** -19 + 2.0 ** -22)  # as cache_ref.attend
    if n_seen is not None:
        hidden = torch.arange(n)[None] >= torch.as_tensor(n_seen)[:, None]
        s = s.masked_fill(hidden[:, None, None], -float("inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("mhgn,nhd->mhgd", p, v)
    size = torch.einsum("mhgn,nhd->mhgd", p, v.abs())
    return out.reshape(m, Hq, D), size.reshape(m, Hq, D), lse.reshape(m, Hq), err


def check(out, lse, ref, n, r, dtype, what="", vmax=0.0):
    """out [m, Hq, D] and lse [m, Hq] against ref = attend_many's result; vmax:
    the largest |v| where weights are f16."""
    o, size, l, err = ref
    bound = size * (r + 4 * err + n * 2.0 ** -23 + 2.0 ** -18) + n * 2.0 ** -24 * vmax
    bound = bound + rounding(o.abs() + bound, dtype)
    off = (out.double() - o).abs()
    assert bool((off <= bound).all()), f"{what}: out off by {float((off - bound).max())} beyond its bound"
    if lse is None:
        return
    empty = torch.isinf(l)
    assert bool((torch.isneginf(lse) == empty).all()), f"{what}: -inf rows of lse"
    loff = (lse.double() - l)[~empty].abs()
    lb = 2 * err + n * 2.0 ** -24 + 2.0 ** -18 * (1 + l[~empty].abs())
    assert bool((loff <= lb).all()), f"{what}: lse off by {float((loff - lb).max())} beyond its bound"


class Cross:
    """A seeded case of cross attention (CPU tensors)."""

    def __init__(self, seed, kv_lens, beams=1, T=1, Hq=4, Hkv=2, D=64, ps=16, kv=torch.bfloat16, q=None, q_lens=None,
                 pad_cols=0, q_mult=1.5, wide=False):
        gen = torch.Generator().manual_seed(seed)
        self.q_dtype = q or (kv if kv != torch.float8_e4m3fn else torch.bfloat16)
        self.kv_lens, self.beams, self.T, self.ps, self.kv = list(kv_lens), beams, T, ps, kv
        B = len(self.kv_lens) * beams
        self.table, pages, _ = make_table(gen, self.kv_lens, ps, extra=2, pad_cols=pad_cols)
        self.k, self.ks, self.v, self.vs = pools(gen, [(self.kv_lens, self.table)], pages, ps, Hkv, D, kv, wide)
        self.wide = wide
        self.q = (q_mult * torch.randn((B, T, Hq, D), generator=gen)).to(self.q_dtype)
        self.q_lens = None if q_lens is None else list(q_lens)

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        mv = lambda t: None if t is None else t.cuda()  # noqa: E731
        return dict(q=self.q.cuda(), k_pages=self.k.cuda(), v_pages=self.v.cuda(), block_table=self.table.cuda(),
                    kv_lens=torch.tensor(self.kv_lens, **i32), k_scale=mv(self.ks), v_scale=mv(self.vs),
                    q_lens=None if self.q_lens is None else torch.tensor(self.q_lens, **i32))

    def verify(self, out, lse, untouched=None, what=""):
        """out [B, T, Hq, D], lse [B, T, Hq]; untouched: the value that rows past q_lens still hold."""
        out, lse = out.cpu(), None if lse is None else lse.cpu()
        k, v = values(self.k, self.ks), values(self.v, self.vs)
        for r, L in enumerate(self.kv_lens):
            kk, vv = seq_tokens(k, self.table[r], L, self.ps), seq_tokens(v, self.table[r], L, self.ps)
            for b in range(r * self.beams, (r + 1) * self.beams):
                n = self.T if self.q_lens is None else self.q_lens[b]
                if n:
                    ref = attend_many(self.q[b, :n].double(), kk, vv)
                    check(out[b, :n], None if lse is None else lse[b, :n], ref, L,
                          r_p(self.q_dtype, self.kv, self.wide), self.q_dtype, what=f"{what} sequence {b}, length {L}",
                          vmax=float(vv.abs().max()) if L and self.kv != torch.bfloat16 else 0.0)
                if untouched is not None and n < self.T:
                    assert bool((out[b, n:] == untouched).all()) and bool((lse[b, n:] == untouched).all()), (what, b)


class Prefix:
    """A seeded case of decode behind shared prefixes (CPU tensors)."""

    def __init__(self, seed, prefix_lens, prefix_of, lens, T=1, Hq=4, Hkv=2, D=64, ps=16, kv=torch.bfloat16, q=None,
                 q_mult=1.5):
        gen = torch.Generator().manual_seed(seed)
        self.q_dtype = q or (kv if kv != torch.float8_e4m3fn else torch.bfloat16)
        self.plens, self.of, self.lens, self.T, self.ps, self.kv = list(prefix_lens), list(prefix_of), list(lens), T, ps, kv
        table, pages, _ = make_table(gen, self.plens + self.lens, ps, extra=2)
        P = len(self.plens)
        cols = lambda ls: max(1, max(-(-n // ps) for n in ls))  # noqa: E731
        self.ptable, self.table = table[:P, :cols(self.plens)].contiguous(), table[P:, :cols(self.lens)].contiguous()
        self.k, self.ks, self.v, self.vs = pools(gen, [(self.plens, self.ptable), (self.lens, self.table)], pages, ps, Hkv,
                                                 D, kv)
        self.q = (q_mult * torch.randn((len(self.lens), T, Hq, D), generator=gen)).to(self.q_dtype)

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        mv = lambda t: None if t is None else t.cuda()  # noqa: E731
        q = self.q.cuda() if self.T > 1 else self.q[:, 0].contiguous().cuda()
        return dict(q=q, k_pages=self.k.cuda(), v_pages=self.v.cuda(), prefix_table=self.ptable.cuda(),
                    prefix_lens=torch.tensor(self.plens, **i32), block_table=self.table.cuda(),
                    seq_lens=torch.tensor(self.lens, **i32), k_scale=mv(self.ks), v_scale=mv(self.vs))

    def verify(self, out, lse, what=""):
        shape = self.q.shape
        out, lse = out.cpu().reshape(shape), None if lse is None else lse.cpu().reshape(shape[:-1])
        k, v = values(self.k, self.ks), values(self.v, self.vs)
        narrow = self.kv != torch.bfloat16  # the own pass works in f16
        r = max(r_p(self.q_dtype, self.kv), 2.0 ** -11)
        for b, L in enumerate(self.lens):
            kk, vv = seq_tokens(k, self.table[b], L, self.ps), seq_tokens(v, self.table[b], L, self.ps)
            if self.of[b] >= 0:
                p = self.of[b]
                kk = torch.cat([seq_tokens(k, self.ptable[p], self.plens[p], self.ps), kk])
                vv = torch.cat([seq_tokens(v, self.ptable[p], self.plens[p], self.ps), vv])
            seen = [kk.shape[0] - self.T + 1 + t for t in range(self.T)]
            ref = attend_many(self.q[b].double(), kk, vv, seen)
            check(out[b], None if lse is None else lse[b], ref, kk.shape[0], r, self.q_dtype,
                  what=f"{what} sequence {b}",
                  vmax=float(vv.abs().max()) if len(vv) and narrow else 0.0)
