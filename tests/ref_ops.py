"""Plain 64-bit forms of the operators around the attention, for the tests: written
from their definitions, element by element where that is what the definition says."""
import math

import torch


def angles(positions, inv_freq):
    return positions.double()[..., None] * inv_freq.double()                # [B, L, F]


def rotate(y, positions, inv_freq, rot_start, interleaved, sign=1.0):
    """y [B, L, H, D] (double) with its pairs turned by sign * angle."""
    F = inv_freq.numel()
    a = angles(positions, inv_freq)[:, :, None, :] * sign
    i = torch.arange(F, device=y.device)
    ia = rot_start + (2 * i if interleaved else i)
    ib = ia + (1 if interleaved else F)
    out = y.clone()
    out[..., ia] = y[..., ia] * a.cos() - y[..., ib] * a.sin()
    out[..., ib] = y[..., ib] * a.cos() + y[..., ia] * a.sin()
    return out


def norm(x, kind, norm_dim, weight, bias, eps):
    """(z, xhat, r) in double; z is x behind norm_dim."""
    if kind is None:
        return x, None, None
    n = x[..., :norm_dim]
    if kind == "layer":
        n = n - n.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((n * n).mean(-1, keepdim=True) + eps)
    xhat = n * r
    z = xhat * weight.double()
    if bias is not None:
        z = z + bias.double()
    return torch.cat((z, x[..., norm_dim:]), -1), xhat, r


def norm_rope(x, positions, inv_freq=None, weight=None, bias=None, kind=None, norm_dim=0, eps=1e-6, rot_start=0,
              interleaved=False):
    z, _, _ = norm(x.double(), kind, norm_dim, weight, bias, eps)
    y = z if inv_freq is None else rotate(z, positions, inv_freq, rot_start, interleaved)
    return y, z


def norm_rope_bwd(dy, x, positions, inv_freq=None, weight=None, bias=None, kind=None, norm_dim=0, eps=1e-6,
                  rot_start=0, interleaved=False):
    """dx, dw, db and the magnitudes their tolerances are made of."""
    dz = dy.double()
    if inv_freq is not None:
        dz = rotate(dz, positions, inv_freq, rot_start, interleaved, -1.0)
    if kind is None:
        return dz, None, None, dict(dx=torch.zeros_like(dz))
    _, xhat, r = norm(x.double(), kind, norm_dim, weight, bias, eps)
    dn = dz[..., :norm_dim]
    g = dn * weight.double()
    dx = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(-1, keepdim=True)
    dx = torch.cat((dx * r, dz[..., norm_dim:]), -1)
    size = r * g.abs().amax(-1, keepdim=True) * (2.0 + math.sqrt(norm_dim))
    size = torch.cat((size.expand_as(dn), torch.zeros_like(dz[..., norm_dim:])), -1)
    rows = (0, 1, 2)
    return dx, (dn * xhat).sum(rows), dn.sum(rows), dict(dx=size, dw=(dn * xhat).abs().sum(rows),
                                                         db=dn.abs().sum(rows))


# ---------------------------------------------------------------- 4-bit cache
def kv4_nibble(d_v, col):
    """(byte, shift) of value column `col` in a cache row."""
    c, part, word, e = col // 64, col // 16 % 4, col // 8 % 2, col % 8
    n = e // 2 + 4 * (e % 2)
    return part * (d_v // 8) + c * 8 + word * 4 + n // 2, 4 * (n % 2)


def kv4_scale_slot(d_v, col):
    g = col // 32
    return (g % 2) * (d_v // 64) + g // 2


def kv4_tables(d_v, device):
    byte, shift = zip(*(kv4_nibble(d_v, c) for c in range(d_v)))
    slot = [kv4_scale_slot(d_v, c) for c in range(d_v)]
    return [torch.tensor(v, device=device) for v in (byte, shift, slot)]


def kv4_values(codes, scales, tail):
    """Rows [..., d_qk] in double from the cache arrays [..., d_v/2], [..., d_v/32], [..., tail]."""
    byte, shift, slot = kv4_tables(2 * codes.shape[-1], codes.device)
    q = ((codes.long()[..., byte] >> shift) & 15) - 8
    return torch.cat((q.double() * scales.double()[..., slot], tail.double()), -1)


def kv4_quantised(kv, d_v):
    """(values [..., d_qk], steps [..., d_v/32]) that the cache holds for bf16 rows, in double."""
    x = kv[..., :d_v].double().unflatten(-1, (-1, 32))
    most = x.abs().amax(-1, keepdim=True)
    need = most / torch.full_like(most, 7.0)
    unit = (need.clamp_min(1e-300).view(torch.int64) & (0x7FF << 52)).view(torch.float64) / 16.0
    step = torch.ceil(need / unit) * unit                                   # five significant bits
    q = (x / step).round()
    zero = most < 2.0 ** -100
    bad = ~(most <= 2.0 ** 126) | ~torch.isfinite(x).all(-1, keepdim=True)
    step = torch.where(zero, 0.0, step)
    step = torch.where(bad, math.nan, step)
    v = torch.where(zero, 0.0, q * step)
    return torch.cat((v.flatten(-2), kv[..., d_v:].double()), -1), step.squeeze(-1)


# ---------------------------------------------------------------- attention
def attention(q, rows, valid, d_v, scale):
    """q [n, H, D]; rows [n, m, D]; valid [n, m]: (out [n, H, d_v], lse [n, H], p [n, H, m]) in double."""
    z = torch.einsum("nhd,nmd->nhm", q.double(), rows.double()) * scale
    z = z.masked_fill(~valid[:, None], -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse.clamp_min(-1e300)[..., None])
    p = torch.where(valid[:, None], p, 0.0)
    v = torch.where(valid[..., None], rows[..., :d_v].double(), 0.0)
    return torch.einsum("nhm,nmd->nhd", p, v), lse, p


def attention_tolerance(q, rows, valid, out, lse, p, d_v, scale):
    """(tolerance of out, of lse) of a bf16 attention against the 64-bit one.

    A logit is a sum of D products in fp32, in any order: off by at most D 2^-24 times the
    sum of their magnitudes, times the scale; call the largest of a row delta (the exponential
    and the row sum add 2^-20).  lse is off by at most delta + 2^-20 (1 + |lse|).
    The output: every probability off by 2 delta of itself and rounded to bf16 once before
    the product with the values (2^-8), the normaliser summed from the unrounded ones, the
    result rounded once (2^-8 of it)."""
    v = torch.where(valid[..., None], rows[..., :d_v].double(), 0.0).abs()
    k = torch.where(valid[..., None], rows.double(), 0.0).abs()
    size = torch.einsum("nhd,nmd->nhm", q.double().abs(), k).amax(-1) * scale
    delta = q.shape[-1] * 2.0 ** -24 * size
    far = 2.0 ** -8 + 2.0 ** -19 + 2 * delta[..., None]
    tol = 2.0 ** -8 * out.abs() + far * torch.einsum("nhm,nmd->nhd", p, v) + 1e-30
    return tol, delta + 2.0 ** -20 * (1 + torch.nan_to_num(lse, neginf=0.0).abs())
