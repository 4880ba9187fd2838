"""Plain float64 definitions of the cache operators (append_kv_norm, the
attention weights, evict_kv, differential attention) on CPU tensors, with the
error bounds the tests hold the kernels to.

Roundings: half a step of the stored type is eps / 2 relative (bf16 2^-8, f16
2^-11, E4M3 2^-4), plus half a subnormal step (f16 2^-25, E4M3 2^-10; bf16's
is below fp32's tiny values).
"""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
             torch.float8_e4m3fn: 2.0 ** -4}
HALF_TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0, torch.float8_e4m3fn: 2.0 ** -10}


def rounding(ref, dtype):
    return HALF_STEP[dtype] * ref.abs() + HALF_TINY[dtype]


def make_pool(gen, pages, ps, H, D, dtype):
    x = torch.randn((pages, ps, H, D), generator=gen)
    if dtype != torch.float8_e4m3fn:
        return x.to(dtype), None
    scale = x.abs().amax(dim=(1, 3)) / 448.0 * (1 + torch.rand((pages, H), generator=gen))
    return (x / scale[:, None, :, None]).to(dtype), scale


def values(pool, scale):
    x = pool.to(torch.float32).double()
    return x if scale is None else x * scale.double()[:, None, :, None]


def make_table(gen, lens, ps, extra=1, pad_cols=0):
    """Random distinct pages for every sequence (-1 past its end); pages in all."""
    need = [-(-int(n) // ps) for n in lens]
    total = sum(need) + extra
    perm = torch.randperm(total, generator=gen).to(torch.int32)
    bt = torch.full((len(lens), max([1] + need) + pad_cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, total, perm[at:]


def norm_rotate(x, w, eps, cos, sin, interleaved):
    """x [n, H, D] float64; cos, sin [n, rd / 2] or None.  Returns the exact
    result and a bound on what fp32 steps move it by: 16 rounding steps of
    2^-24 (12 for the sum of squares and rsqrt, halved by the square root but
    doubled for rsqrt's own 2 ulp; 3 for the products; 1 for the sum) on the
    terms that are added, taken as 2^-20."""
    y = x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    size = y.abs()
    if cos is not None:
        rd = 2 * cos.shape[-1]
        i = torch.arange(rd // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
        c, s = cos.double()[:, None], sin.double()[:, None]
        z, zs = y.clone(), size.clone()
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        zs[..., a] = size[..., a] * c.abs() + size[..., b] * s.abs()
        zs[..., b] = size[..., b] * c.abs() + size[..., a] * s.abs()
        y, size = z, zs
    return y, size * 2.0 ** -20


def seq_tokens(vals, table_row, L, ps):
    """[L, H, D] of a block-table row."""
    ids = table_row[:-(-L // ps)].long()
    return vals[ids].flatten(0, 1)[:L]


def attend(q, k, n, width, off):
    """Scores of q [Hkv, G, D] over k [n, Hkv, D], elements [off, off + width):
    probabilities, lse and a bound on a score's error.  The product sums width
    terms in fp32 on the tensor cores: at most 8 steps, each off by 2^-22 of
    the terms' magnitudes, then the scaling by a rounded factor (2^-22 of the
    score)."""
    scale = width ** -0.5
    qq, kk = q[..., off:off + width], k[:n, :, off:off + width]
    s = torch.einsum("hgd,nhd->hgn", qq, kk) * scale
    mag = torch.einsum("hgd,nhd->hgn", qq.abs(), kk.abs()) * scale
    err = float(mag.max()) * (2.0 ** -19 + 2.0 ** -22) if n else 0.0
    lse = torch.logsumexp(s, -1) if n else torch.full(s.shape[:2], -float("inf"), dtype=torch.float64)
    p = torch.exp(s - lse[..., None]) if n else s
    return p, lse, err


def evict(weights_row, L, budget, sinks, recent):
    """Indices that stay of one (sequence, KV head): weights_row [N] fp32."""
    if L <= budget:
        return torch.arange(L)
    mid = torch.arange(sinks, L - recent)
    many = budget - sinks - recent
    w = weights_row[mid].double()
    w = torch.where(torch.isnan(w), torch.full_like(w, -float("inf")), w)
    nan = torch.isnan(weights_row[mid])
    # stable: NaN below -inf, equal weights lowest index first
    order = sorted(range(len(mid)), key=lambda i: (bool(nan[i]), -float(w[i])))[:many]
    return torch.cat([torch.arange(sinks), mid[sorted(order)], torch.arange(L - recent, L)])
