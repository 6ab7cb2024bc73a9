"""Measured cases of the operators around the sparse attention: the norm and
rotation that make queries and keys, the 4-bit latent cache, attention over that
cache, and attention with a sliding window and sinks.

`run` computes a case in its plain form (elementary torch operations in 32 bits)
or, where `own` is true, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
SCALE = 1.0 / math.sqrt(192.0)      # the softmax scale of the repository's workloads
THETA = 10000.0

# (H, d_qk, d_v) of the latent attention; "mla" is the model shape of the benchmark's
# workloads, "tiny" that of the tiny workload
SHAPES = {"mla": (128, 576, 512), "tiny": (16, 192, 128)}


def listed():
    return [
        # one new token for each of 64 sequences: the indexer's queries, per-head RMS norm, e4m3 for the indexer
        dict(name="norm_rope decode q_I", op="norm_rope", B=64, L=1, H=64, D=128, norm="rms", norm_dim=128,
             rot_start=0, rot_dim=64, interleaved=False, e4m3=True),
        # the indexer's keys of a 32K prompt: layer norm with bias, one head
        dict(name="norm_rope 32K k_I", op="norm_rope", B=1, L=32768, H=1, D=128, norm="layer", norm_dim=128,
             rot_start=0, rot_dim=64, interleaved=False, e4m3=True),
        # the indexer's queries of an 8K prompt
        dict(name="norm_rope 8K q_I", op="norm_rope", B=1, L=8192, H=64, D=128, norm="rms", norm_dim=128,
             rot_start=0, rot_dim=64, interleaved=False, e4m3=True),
        # attention queries of a 4096-token chunk, rotated behind 128 plain columns, in bf16
        dict(name="norm_rope 4K q", op="norm_rope", B=1, L=4096, H=128, D=192, norm="rms", norm_dim=128,
             rot_start=128, rot_dim=64, interleaved=True, e4m3=False),
        # training the indexer on a 4096-token chunk: gradient of its queries' norm and rotation
        dict(name="norm_rope_bwd 4K q_I", op="norm_rope_bwd", B=1, L=4096, H=64, D=128, norm="rms", norm_dim=128,
             rot_start=0, rot_dim=64, interleaved=False),
        # the same for its keys: two ragged sequences, layer norm, one head
        dict(name="norm_rope_bwd 8K k_I", op="norm_rope_bwd", B=2, L=8191, H=1, D=128, norm="layer", norm_dim=128,
             rot_start=0, rot_dim=64, interleaved=False),
        # one new latent row for each of 64 sequences of different lengths goes into the cache
        dict(name="kv4 store decode", op="kv4_store", shape="mla", B=64, L=1, Lk=1024),
        # a 32K prompt's latent rows go into the cache
        dict(name="kv4 store 32K", op="kv4_store", shape="mla", B=1, L=32768, Lk=32800),
        # decode: 64 sequences, 2048 selected rows each out of 32K cached ones
        dict(name="sparse_attn_kv4 decode", op="sparse_attn_kv4", shape="mla", B=64, Lq=1, Lk=32768, k=2048),
        # a chunk of 1024 queries over a 32K cache
        dict(name="sparse_attn_kv4 chunk", op="sparse_attn_kv4", shape="mla", B=1, Lq=1024, Lk=32768, k=2048),
        # decode in a window layer: 32 sequences of different lengths, 1024 recent rows and 4 sinks
        dict(name="window_attn decode", op="window_attn", shape="mla", B=32, Lq=1, Lk=8192, window=1024, sinks=4),
        # a prompt through a window layer
        dict(name="window_attn prefill", op="window_attn", shape="mla", B=1, Lq=4096, Lk=4096, window=512, sinks=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "kv4_store", "sparse_attn_kv4", "window_attn"])
    if op in ("norm_rope", "norm_rope_bwd"):
        H, D, nd, rs, rd = rng.choice([(64, 128, 128, 0, 64), (1, 128, 128, 0, 64), (128, 192, 128, 128, 64),
                                       (1, 576, 512, 512, 64), (4, 64, 64, 0, 64), (16, 192, 192, 64, 128),
                                       (1, 64, 64, 0, 32)])
        B = rng.choice([1, 1, 2, 3, 7])
        L = max(1, _log(rng, 1, 4.0e6 if op == "norm_rope_bwd" else 8.0e6) // (B * H * D // 8))
        case = dict(op=op, B=B, L=L, H=H, D=D, norm=rng.choice(["rms", "rms", "layer"]), norm_dim=nd, rot_start=rs,
                    rot_dim=rd, interleaved=rng.random() < 0.5)
        if op == "norm_rope":
            case["e4m3"] = rng.random() < 0.5
        return case
    shape = rng.choice(["mla", "mla", "mla", "tiny"])
    if op == "kv4_store":
        B = rng.choice([1, 3, 16, 64])
        L = max(1, _log(rng, 1, 32768) // B)
        return dict(op=op, shape=shape, B=B, L=L, Lk=L + rng.randrange(0, 700))
    decode = rng.random() < 0.5
    B, Lq = (_log(rng, 1, 64), rng.choice([1, 1, 2])) if decode else (rng.choice([1, 2]), _log(rng, 3, 500))
    if op == "sparse_attn_kv4":
        Lk = Lq + _log(rng, 40, 16384)
        return dict(op=op, shape=shape, B=B, Lq=Lq, Lk=Lk, k=min(2048, _log(rng, 16, 2600)))
    Lk = Lq + (_log(rng, 1, 8192) if decode else rng.choice([0, _log(rng, 1, 4096)]))
    return dict(op=op, shape=shape, B=B, Lq=Lq, Lk=Lk, window=_log(rng, 1, 2048), sinks=rng.choice([0, 1, 4, 16, 130]))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _order(d_v):
    """The column that each nibble of a cache row holds: row byte (part, chunk, word, byte), low nibble first."""
    n = d_v // 64
    part, chunk, word, byte, nib = torch.meshgrid(torch.arange(4), torch.arange(n), torch.arange(2), torch.arange(4),
                                                  torch.arange(2), indexing="ij")
    return (chunk * 64 + part * 16 + word * 8 + (byte % 2) * 4 + nib * 2 + byte // 2).reshape(-1).to(DEV)


def _scale_order(d_v):
    """The 32-column group that each scale of a cache row belongs to: (half, chunk)."""
    half, chunk = torch.meshgrid(torch.arange(2), torch.arange(d_v // 64), indexing="ij")
    return (chunk * 2 + half).reshape(-1).to(DEV)


def _random_cache(g, B, Lk, d_qk, d_v):
    """A cache as a program has it: Gaussian latents in groups of 32, each with its scale."""
    q = _randn(g, B, Lk, d_v).mul_(2.9).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    q = q[..., _order(d_v)]
    codes = q[..., 0::2] | (q[..., 1::2] << 4)
    scales = torch.randint(16, 32, (B, Lk, d_v // 32), generator=g, device=DEV).to(torch.bfloat16) / 64
    return codes.contiguous(), scales, _randn(g, B, Lk, d_qk - d_v)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm_rope", "norm_rope_bwd"):
        B, L, H, D, nd = (case[x] for x in ("B", "L", "H", "D", "norm_dim"))
        s["x"] = _randn(g, B, L, H, D)
        s["weight"] = 1 + 0.1 * torch.randn(nd, generator=g, device=DEV)
        s["bias"] = 0.1 * torch.randn(nd, generator=g, device=DEV) if case["norm"] == "layer" else None
        s["inv_freq"] = THETA ** (-torch.arange(0, case["rot_dim"], 2, device=DEV, dtype=torch.float64)
                                  / case["rot_dim"])
        s["inv_freq"] = s["inv_freq"].float()
        # each sequence goes on from a place of its own
        first = torch.randint(0, 100000, (B, 1), generator=g, device=DEV, dtype=torch.int32)
        s["positions"] = first + torch.arange(L, device=DEV, dtype=torch.int32)
        if op == "norm_rope_bwd":
            s["dy"] = _randn(g, B, L, H, D)
        return s
    H, d_qk, d_v = SHAPES[case["shape"]]
    B, Lk = case["B"], case["Lk"]
    if op == "kv4_store":
        s["kv"] = _randn(g, B, case["L"], d_qk)
        s["start"] = torch.randint(0, Lk - case["L"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["codes"] = torch.zeros(B, Lk, d_v // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(B, Lk, d_v // 32, dtype=torch.bfloat16, device=DEV)
        s["tail"] = torch.zeros(B, Lk, d_qk - d_v, dtype=torch.bfloat16, device=DEV)
        return s
    Lq = case["Lq"]
    s["q"] = _randn(g, B, Lq, H, d_qk)
    if op == "sparse_attn_kv4":
        s["codes"], s["scales"], s["tail"] = _random_cache(g, B, Lk, d_qk, d_v)
        # what the selection returns: distinct positions up to the query's own, ascending, -1 behind them
        t = torch.arange(Lk - Lq, Lk, device=DEV).view(1, Lq, 1)
        pos = torch.arange(Lk, device=DEV)
        score = torch.rand(B, Lq, Lk, generator=g, device=DEV).masked_fill_(pos > t, -1.0)
        n = min(case["k"], Lk)
        top, idx = score.topk(n, dim=-1)
        idx = torch.where(top >= 0, idx, Lk).sort(dim=-1).values
        s["indices"] = torch.full((B, Lq, case["k"]), -1, dtype=torch.int32, device=DEV)
        s["indices"][..., :n] = torch.where(idx < Lk, idx, -1)
        return s
    s["kv"] = _randn(g, B, Lk, d_qk)
    s["start"] = torch.randint(0, Lk - Lq + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    if B == 1:
        s["start"].fill_(Lk - Lq)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _cos_sin(s, dtype=torch.float32):
    a = s["positions"].double().unsqueeze(-1) * s["inv_freq"].double()       # far positions: angles in 64 bits
    return a.cos().to(dtype).unsqueeze(2), a.sin().to(dtype).unsqueeze(2)    # [B, L, 1, rot_dim/2]


def _pairs(s, x):
    r = x[..., s["rot_start"]:s["rot_start"] + s["rot_dim"]]
    if s["interleaved"]:
        return r[..., 0::2], r[..., 1::2]
    return r.chunk(2, dim=-1)


def _rotate(s, x, sign):
    c, sn = _cos_sin(s)
    a, b = _pairs(s, x)
    ra, rb = a * c - sign * b * sn, b * c + sign * a * sn
    rot = torch.stack((ra, rb), dim=-1).flatten(-2) if s["interleaved"] else torch.cat((ra, rb), dim=-1)
    lo, hi = s["rot_start"], s["rot_start"] + s["rot_dim"]
    return torch.cat((x[..., :lo], rot, x[..., hi:]), dim=-1)


EPS = 1e-6


def _normed(s, x):
    n = x[..., :s["norm_dim"]]
    if s["norm"] == "layer":
        n = n - n.mean(dim=-1, keepdim=True)
    r = (n.square().mean(dim=-1, keepdim=True) + EPS).rsqrt()
    return n * r, r


def _plain_norm_rope(s):
    x = s["x"].float()
    xhat, _ = _normed(s, x)
    z = xhat * s["weight"]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _rotate(s, torch.cat((z, x[..., s["norm_dim"]:]), dim=-1), 1.0)
    if not s["e4m3"]:
        return y.to(torch.bfloat16)
    scale = y.abs().amax(dim=(-2, -1)).clamp_min(1e-30) / 448.0
    codes = (y / scale[..., None, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, scale


def _plain_norm_rope_bwd(s):
    x = s["x"].float()
    dz = _rotate(s, s["dy"].float(), -1.0)
    nd = s["norm_dim"]
    xhat, r = _normed(s, x)
    dn = dz[..., :nd]
    dxhat = dn * s["weight"]
    dx = dxhat - xhat * (dxhat * xhat).mean(dim=-1, keepdim=True)
    if s["norm"] == "layer":
        dx = dx - dxhat.mean(dim=-1, keepdim=True)
    dx = torch.cat((dx * r, dz[..., nd:]), dim=-1).to(torch.bfloat16)
    dw = (dn * xhat).sum(dim=(0, 1, 2))
    return [dx, dw] + ([dn.sum(dim=(0, 1, 2))] if s["bias"] is not None else [])


def _plain_kv4_store(s):
    d_v = s["codes"].shape[-1] * 2
    kv = s["kv"]
    x = kv[..., :d_v].float().unflatten(-1, (-1, 32))
    most = x.abs().amax(dim=-1, keepdim=True)
    bits = (most / torch.full_like(most, 7.0)).view(torch.int32)
    step = ((bits + 0x7FFFF) & -0x80000).view(torch.float32)         # five significant bits, rounded up
    q = torch.where(step > 0, (x / step).round(), 0.0)
    rows = s["start"].long().unsqueeze(1) + torch.arange(kv.shape[1], device=DEV)
    at = torch.arange(kv.shape[0], device=DEV).unsqueeze(1)
    nib = (q.flatten(-2) + 8).to(torch.uint8)[..., _order(d_v)]
    s["codes"][at, rows] = nib[..., 0::2] | (nib[..., 1::2] << 4)
    s["scales"][at, rows] = step.squeeze(-1)[..., _scale_order(d_v)].to(torch.bfloat16)
    s["tail"][at, rows] = kv[..., d_v:]
    return torch.cat(((q * step).flatten(-2).to(torch.bfloat16), kv[..., d_v:]), dim=-1), s["scales"], s["tail"]


def _unpacked(codes, scales, tail):
    """fp32 latent rows [..., d_qk] of cache rows."""
    n = codes.shape[-1] // 32
    v = torch.stack((codes & 15, codes >> 4), dim=-1).float() - 8.0
    v = v.unflatten(-2, (4, n, 2, 2, 2))                              # part, chunk, word, odd, quarter | nibble
    k = v.dim()
    lead = list(range(k - 6))
    v = v.permute(*lead, k - 5, k - 6, k - 4, k - 2, k - 1, k - 3).flatten(-6)
    st = scales.float().unflatten(-1, (2, n)).transpose(-1, -2).flatten(-2)
    return torch.cat(((v.unflatten(-1, (-1, 32)) * st.unsqueeze(-1)).flatten(-2), tail.float()), dim=-1)


def _attend(q, rows, valid, d_v):
    """q [B, Lq, H, D], rows [B, Lq, n, D] fp32, valid [B, Lq, n]; a row with nothing to see gives 0 and -inf."""
    z = (q.float() * SCALE) @ rows.transpose(-1, -2)
    z = z.masked_fill(~valid.unsqueeze(2), -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = (z - m.clamp_min(-3.0e38)).exp()
    total = p.sum(dim=-1, keepdim=True)
    out = p @ rows[..., :d_v] / total.clamp_min(1e-38)
    return out.to(torch.bfloat16), (m + total.log()).squeeze(-1)


def _plain_sparse_attn_kv4(s):
    idx = s["indices"].long()
    valid = idx >= 0
    idx = idx.clamp_min(0)
    at = torch.arange(idx.shape[0], device=DEV).view(-1, 1, 1)
    rows = _unpacked(s["codes"][at, idx], s["scales"][at, idx], s["tail"][at, idx])
    return _attend(s["q"], rows, valid, s["codes"].shape[-1] * 2)


def _window_rows(s):
    """Positions that each query sees, [B, Lq, n], and which of them are there."""
    Lq = s["q"].shape[1]
    t = (s["start"].long().unsqueeze(1) + torch.arange(Lq, device=DEV)).unsqueeze(-1)
    lo = (t - s["window"] + 1).clamp_min(0)
    w = lo + torch.arange(min(s["window"], s["kv"].shape[1]), device=DEV)
    sk = torch.arange(min(s["sinks"], s["kv"].shape[1]), device=DEV).expand(*t.shape[:2], -1)
    pos = torch.cat((sk, w), dim=-1)
    return pos, torch.cat((sk < lo, w <= t), dim=-1)


def _plain_window_attn(s):
    pos, valid = _window_rows(s)
    at = torch.arange(pos.shape[0], device=DEV).view(-1, 1, 1)
    rows = s["kv"][at, pos.clamp_max(s["kv"].shape[1] - 1)].float()
    return _attend(s["q"], rows, valid, SHAPES[s["shape"]][2])


PLAIN = {"norm_rope": _plain_norm_rope, "norm_rope_bwd": _plain_norm_rope_bwd, "kv4_store": _plain_kv4_store,
         "sparse_attn_kv4": _plain_sparse_attn_kv4, "window_attn": _plain_window_attn}


# ---------------------------------------------------------------- the library's entry points
def _own(s):
    import sparse_attention_19_b200 as dsa
    op = s["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        how = dict(weight=s["weight"], bias=s["bias"], norm=s["norm"], norm_dim=s["norm_dim"], eps=EPS,
                   rot_start=s["rot_start"], interleaved=s["interleaved"], positions=s["positions"])
        if op == "norm_rope":
            return dsa.norm_rope(s["x"], s["inv_freq"], e4m3=s["e4m3"], **how)
        return [g for g in dsa.norm_rope_bwd(s["dy"], s["x"], s["inv_freq"], **how) if g is not None]
    if op == "kv4_store":
        dsa.kv4_write(s["kv"], s["codes"], s["scales"], s["tail"], start=s["start"])
        rows = dsa.kv4_read(s["codes"], s["scales"], s["tail"], s["kv"].shape[1], start=s["start"])
        return rows, s["scales"], s["tail"]
    if op == "sparse_attn_kv4":
        return dsa.sparse_attn_kv4(s["q"], s["codes"], s["scales"], s["tail"], s["indices"], SCALE)
    return dsa.window_attn(s["q"], s["kv"], SHAPES[s["shape"]][2], SCALE, s["window"], s["sinks"], start=s["start"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        n = case["B"] * case["L"] * case["H"] * case["D"]
        if op == "norm_rope_bwd":
            return dict(bytes=6 * n, flops=20 * n)
        return dict(bytes=2 * n + (n if case["e4m3"] else 2 * n), flops=10 * n)
    H, d_qk, d_v = SHAPES[case["shape"]]
    row4 = d_v // 2 + d_v // 16 + 2 * (d_qk - d_v)
    B = case["B"]
    if op == "kv4_store":
        return dict(bytes=B * case["L"] * (4 * d_qk + row4), flops=4 * B * case["L"] * d_v)
    Lq, Lk = case["Lq"], case["Lk"]
    ends = range(Lk - Lq + 1, Lk + 1)
    if op == "sparse_attn_kv4":
        pairs = B * sum(min(case["k"], e) for e in ends)
        rows, width = B * min(Lk, Lq * min(case["k"], Lk)), row4
        read = B * Lq * case["k"] * 4
    else:
        n = case["window"] + case["sinks"]
        pairs = B * sum(min(n, e) for e in ends)
        rows, width = B * min(Lk, Lq + n), 2 * d_qk
        read = 4 * B
    return dict(bytes=rows * width + read + B * Lq * H * (2 * d_qk + 2 * d_v + 4), flops=2 * H * (d_qk + d_v) * pairs)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_angles(s):
    pos = s["positions"].double()
    return pos[:, :, None, None] * s["inv_freq"].double()


def _exact_norm_rope(s, backward):
    """The head as a chain of linear maps and one norm, in 64 bits; the gradient from autograd on it."""
    x = s["x"].double().requires_grad_(backward)
    w = s["weight"].double().requires_grad_(backward)
    b = s["bias"].double().requires_grad_(backward) if s["bias"] is not None else None
    nd, lo, rd = s["norm_dim"], s["rot_start"], s["rot_dim"]
    head = x[..., :nd]
    if s["norm"] == "layer":
        var, mean = torch.var_mean(head, dim=-1, keepdim=True, unbiased=False)
        head = (head - mean) / torch.sqrt(var + EPS) * w + b
    else:
        head = head / torch.sqrt((head * head).sum(dim=-1, keepdim=True) / nd + EPS) * w
    z = torch.cat((head, x[..., nd:]), dim=-1)
    first = torch.arange(rd // 2, device=DEV) * (2 if s["interleaved"] else 1) + lo
    second = first + (1 if s["interleaved"] else rd // 2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), _exact_angles(s))
    both = torch.complex(z[..., first], z[..., second]) * turn
    y = z.index_copy(-1, torch.cat((first, second)), torch.cat((both.real, both.imag), dim=-1))
    if backward:
        leaves = [x, w] + ([b] if b is not None else [])
        grads = torch.autograd.grad(y, leaves, s["dy"].double())
        return [v.detach() for v in grads]
    if not s["e4m3"]:
        return y
    scale = y.abs().flatten(-2).max(dim=-1).values.clamp_min(1e-30) / 448.0
    return y / scale[..., None, None], scale


def _exact_kv4_store(s):
    d_v = s["codes"].shape[-1] * 2
    x = s["kv"].double()
    groups = x[..., :d_v].reshape(*x.shape[:2], d_v // 32, 32)
    most = groups.abs().max(dim=-1, keepdim=True).values
    need = most / torch.full_like(most, 7.0)
    unit = (need.clamp_min(1e-300).view(torch.int64) & (0x7FF << 52)).view(torch.float64) / 16.0
    step = torch.ceil(need / unit) * unit
    held = torch.where(need > 0, torch.round(groups / step) * step, torch.zeros_like(groups))
    return torch.cat((held.reshape(*x.shape[:2], d_v), x[..., d_v:]), dim=-1), None, None


def _exact_rows(s, at, pos):
    """64-bit latent rows of the 4-bit cache, column by column from the layout's table."""
    d_v = s["codes"].shape[-1] * 2
    bytes_ = s["codes"][at, pos].long()
    nib = torch.empty(*bytes_.shape[:-1], d_v, dtype=torch.float64, device=DEV)
    order = _order(d_v)
    nib[..., order[0::2]] = (bytes_ % 16 - 8).double()
    nib[..., order[1::2]] = (bytes_ // 16 - 8).double()
    st = torch.empty(*bytes_.shape[:-1], d_v // 32, dtype=torch.float64, device=DEV)
    st[..., _scale_order(d_v)] = s["scales"][at, pos].double()
    nib *= st.repeat_interleave(32, dim=-1)
    return torch.cat((nib, s["tail"][at, pos].double()), dim=-1)


def _exact_attend(s, rows, seen, d_v):
    z = torch.einsum("blhd,blnd->blhn", s["q"].double(), rows) * SCALE
    z = torch.where(seen.unsqueeze(2), z, torch.full((), -math.inf, dtype=torch.float64, device=DEV))
    lse = torch.logsumexp(z, dim=-1)
    p = torch.where(seen.unsqueeze(2), torch.exp(z - lse.unsqueeze(-1)), torch.zeros((), dtype=torch.float64, device=DEV))
    return torch.einsum("blhn,blnd->blhd", p, rows[..., :d_v]), lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        return _exact_norm_rope(s, op == "norm_rope_bwd")
    if op == "kv4_store":
        return _exact_kv4_store(s)
    d_v = SHAPES[case["shape"]][2]
    if op == "sparse_attn_kv4":
        pos = s["indices"].long()
        seen = pos >= 0
        at = torch.arange(pos.shape[0], device=DEV)[:, None, None]
        return _exact_attend(s, _exact_rows(s, at, torch.where(seen, pos, 0)), seen, d_v)
    # every cached row against the definition of what a query sees, one query after the other
    B, Lq, H, _ = s["q"].shape
    Lk = s["kv"].shape[1]
    key = torch.arange(Lk, device=DEV)
    kv = s["kv"].double()
    out = torch.empty(B, Lq, H, d_v, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Lq, H, dtype=torch.float64, device=DEV)
    first = s["start"].tolist()
    for b in range(B):
        for i in range(Lq):
            t = first[b] + i
            pos = key[(key <= t) & ((key > t - s["window"]) | (key < s["sinks"]))]
            rows = kv[b].index_select(0, pos)
            z = (s["q"][b, i].double() @ rows.T) * SCALE
            lse[b, i] = torch.logsumexp(z, dim=-1)
            out[b, i] = torch.softmax(z, dim=-1) @ rows[:, :d_v]
    return out, lse
