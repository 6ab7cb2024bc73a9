"""Attention over the 4-bit latent cache against the 64-bit form, and bit for bit against
dsa_sparse_attn over the rows that the cache reads back as (its values are exact in
bf16, and both kernels run the same matrix products over the same tiles)."""
import math

import pytest
import torch

import ref_ops as R
import sparse_attention_19_b200 as dsa
from dsa_inputs import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(192.0)
SHAPES = {"mla": (128, 576, 512), "tiny": (16, 192, 128)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    assert dsa.device_status() == 0


def _cache(kv, d_v):
    cache = dsa.kv4_cache(kv.shape[0], kv.shape[1], kv.shape[2], d_v)
    dsa.kv4_write(kv, *cache)
    return cache


def _inputs(shape, B, Lq, Lk, seed):
    H, D, d_v = SHAPES[shape]
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(B, Lq, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    kv = torch.randn(B, Lk, D, generator=g, device=DEV, dtype=torch.bfloat16)
    return q, kv, d_v, g


def _indices(g, B, Lq, Lk, k, kind):
    if kind == "prefix":                                   # valid entries first, as the top-k writes them
        n = min(k, Lk)
        idx = torch.rand(B, Lq, Lk, generator=g, device=DEV).argsort(-1)[..., :n].sort(-1).values
        out = torch.full((B, Lq, k), -1, device=DEV, dtype=torch.int32)
        out[..., :n] = idx
        return out
    idx = torch.randint(0, Lk, (B, Lq, k), generator=g, device=DEV, dtype=torch.int32)   # repeated entries
    drop = torch.rand(B, Lq, k, generator=g, device=DEV)
    idx[drop < 0.2] = -1
    idx[(drop > 0.2) & (drop < 0.25)] = Lk
    idx[(drop > 0.25) & (drop < 0.3)] = 2 ** 31 - 1
    idx[(drop > 0.3) & (drop < 0.33)] = -(2 ** 31)
    idx[0, 0] = -1                                         # a row with nothing
    return idx


def _check(q, cache, idx, d_v, out, lse, rows=None):
    B, Lq, H, D = q.shape
    n = torch.arange(B * Lq, device=DEV) if rows is None else torch.as_tensor(rows, device=DEV)
    b = n // Lq
    ix = idx.reshape(B * Lq, -1)[n].long()
    Lk = cache[0].shape[1]
    valid = (ix >= 0) & (ix < Lk)
    at = torch.where(valid, ix, 0)
    got_rows = R.kv4_values(*(t[b[:, None], at] for t in cache))
    qq = q.reshape(B * Lq, H, D)[n]
    ro, rl, p = R.attention(qq, got_rows, valid, d_v, SCALE)
    to, tl = R.attention_tolerance(qq, got_rows, valid, ro, rl, p, d_v, SCALE)
    o, l = out.reshape(B * Lq, H, d_v)[n].double(), lse.reshape(B * Lq, H)[n].double()
    assert ((o - ro).abs() <= to).all(), ((o - ro).abs() / to).max()
    none = ~valid.any(-1)
    assert (o[none] == 0).all() and (l[none] == -math.inf).all()
    assert ((l - rl).abs()[~none] <= tl[~none]).all()


@pytest.mark.parametrize("shape", ["mla", "tiny"])
@pytest.mark.parametrize("kind", ["prefix", "holes"])
@pytest.mark.parametrize("B,Lq,Lk,k", [(1, 1, 1, 1), (2, 3, 300, 130), (3, 1, 77, 128), (1, 5, 4000, 2048),
                                       (1, 90, 500, 257), (2, 100, 333, 64), (64, 1, 2500, 2048), (76, 2, 600, 385)])
def test_against_the_64_bit_form(shape, kind, B, Lq, Lk, k):
    q, kv, d_v, g = _inputs(shape, B, Lq, Lk, B * 1000 + k)
    cache = _cache(kv, d_v)
    idx = _indices(g, B, Lq, Lk, k, kind)
    out, lse = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    n = B * Lq
    _check(q, cache, idx, d_v, out, lse, sorted({0, 1 % n, n // 2, n - 1, (7 * n) // 9, 73 % n, 74 % n, 148 % n}))
    # the bf16 attention over what the cache holds
    o2, l2 = dsa.sparse_attn(q, dsa.kv4_read(*cache, Lk), idx, d_v, SCALE)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("shape", ["mla", "tiny"])
def test_rows_that_are_not_selected_may_hold_anything(shape):
    q, kv, d_v, g = _inputs(shape, 2, 40, 900, 3)
    cache = _cache(kv, d_v)
    idx = _indices(g, 2, 40, 900, 200, "holes")
    idx = torch.where(idx % 3 == 1, idx, -1)               # row 0 among those never named
    want = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    bad = torch.arange(900, device=DEV) % 3 != 1
    cache[0][:, bad] = 0
    cache[1][:, bad] = float("nan")
    cache[2][:, bad] = float("inf")
    got = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a NaN in a selected row reaches the rows that select it
    cache[1][0, 4] = float("nan")
    idx[0, 5, 7] = 4
    out, _ = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    assert out[0, 5].isnan().any()


def test_many_units_per_cluster_and_long_rows():
    # 500 rows over 74 cluster pairs: the loaders run across unit boundaries
    q, kv, d_v, g = _inputs("mla", 1, 500, 3000, 5)
    cache = _cache(kv, d_v)
    idx = _indices(g, 1, 500, 3000, 1000, "prefix")
    idx[0, ::7, 100:] = -1
    idx[0, 3::11] = -1
    out, lse = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    _check(q, cache, idx, d_v, out, lse, range(0, 500, 13))
    o2, l2 = dsa.sparse_attn(q, dsa.kv4_read(*cache, 3000), idx, d_v, SCALE)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def _both_ways(q, cache, idx):
    """Over the unpacked rows (the workspace that the binding takes) and in the kernel (the least one)."""
    B, Lq, H, D = q.shape
    d_v = 2 * cache[0].shape[-1]
    Lk, k = cache[0].shape[1], idx.shape[-1]
    assert dsa.workspace_size(dsa.OP_SPARSE_ATTN_KV4, B, Lq, Lk, k, H, d_v) > B * Lk * D * 2, "the rule does not unpack"
    least = max(dsa.workspace_size(dsa.OP_SPARSE_ATTN, B, Lq, max(Lk, Lq), k, H, d_v), 16)
    return (dsa.sparse_attn_kv4(q, *cache, idx, SCALE),
            dsa.sparse_attn_kv4(q, *cache, idx, SCALE, workspace=torch.empty(least, device=DEV, dtype=torch.uint8)))


@pytest.mark.parametrize("shape", ["mla", "tiny"])
@pytest.mark.parametrize("kind", ["prefix", "holes"])
@pytest.mark.parametrize("B,Lq,Lk,k", [(1, 600, 3000, 1000), (3, 200, 1111, 513), (2, 3000, 40, 48), (1, 70, 65, 2048 - 31),
                                       (1, 7, 1, 1)])
def test_unpacked_rows_give_the_same_bits(shape, kind, B, Lq, Lk, k):
    if Lq * Lk * B < 140000:                               # enough slots for the rule
        Lq = 140000 // (B * Lk) + 1
    if shape == "mla" and Lq > 10000:
        pytest.skip("20 GB of queries; the narrow shape covers it")
    q, kv, d_v, g = _inputs(shape, B, Lq, Lk, 17)
    cache = _cache(kv, d_v)
    idx = _indices(g, B, Lq, Lk, k, kind)
    idx[0, 1::13] = -1
    (o, l), (o2, l2) = _both_ways(q, cache, idx)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    n = B * Lq
    _check(q, cache, idx, d_v, o, l, [0, 1, n // 2, n - 1])


@pytest.mark.parametrize("shape", ["mla", "tiny"])
def test_unpacked_rows_that_are_not_selected_may_hold_anything(shape):
    q, kv, d_v, g = _inputs(shape, 2, 400, 900, 3)
    cache = _cache(kv, d_v)
    idx = _indices(g, 2, 400, 900, 300, "holes")
    idx = torch.where(idx % 3 == 1, idx, -1)               # row 0 among those never named
    want = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    bad = torch.arange(900, device=DEV) % 3 != 1
    cache[0][:, bad] = 0
    cache[1][:, bad] = float("nan")
    cache[2][:, bad] = float("inf")
    for o, l in _both_ways(q, cache, idx):
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    # a NaN reaches the queries that select its row and no other
    cache[1][0, 0] = float("nan")
    cache[2][0, 0] = 0
    idx[0, 5, 7] = 0
    for o, _ in _both_ways(q, cache, idx):
        assert o[0, 5].isnan().any()
        hit = torch.zeros(2, 400, dtype=torch.bool, device=DEV)
        hit[0, 5] = True
        assert torch.equal(o[~hit], want[0][~hit])


def test_unpacked_rows_two_calls_at_once_and_from_a_graph():
    q, kv, d_v, g = _inputs("mla", 1, 300, 1500, 9)
    cache, other = _cache(kv, d_v), _cache(kv.flip(1), d_v)
    idx = _indices(g, 1, 300, 1500, 600, "prefix")
    want, want2 = (_both_ways(q, c, idx)[1] for c in (cache, other))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [dsa.sparse_attn_kv4(q, *(other if i % 2 else cache), idx, SCALE, stream=s2 if i % 2 else s1) for i in range(6)]
    s1.synchronize()
    s2.synchronize()
    for i, (o, l) in enumerate(got):
        wo, wl = want2 if i % 2 else want
        assert torch.equal(o, wo) and torch.equal(l, wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    for a, b in zip(cache, other):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want2[0]) and torch.equal(l, want2[1])


@pytest.mark.parametrize("Lq,k", [(200, 1000), (5, 2048), (12, 2048)])
def test_low_memory_takes_no_room_for_unpacked_rows(Lq, k):
    # many rows: no workspace at all; few: the partial results of the splits
    q, kv, d_v, g = _inputs("mla", 1, Lq, 20000 if Lq == 200 else 900, 23)
    cache = _cache(kv, d_v)
    Lk = kv.shape[1]
    idx = _indices(g, 1, Lq, Lk, k, "prefix")
    want = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    least = dsa.workspace_size(dsa.OP_SPARSE_ATTN, 1, Lq, Lk, k, 128, 512)
    assert (least > 0) == (Lq != 200)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    dsa.sparse_attn_kv4(q, *cache, idx, SCALE, out=out, lse=lse, low_memory=True)
    torch.cuda.synchronize()
    # the allocator hands out blocks in steps of 2 MB at most
    assert torch.cuda.max_memory_allocated() - before <= (least + (2 << 20) if least else 0)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_forward_over_unpacked_rows():
    wl = WORKLOADS["prefill_8k"].with_(B=1, Lq=700, Lk=4200, q_offset=3500)
    inp = make_inputs(wl, DEV, 1)
    cache = _cache(inp["kv"], wl.Dv)
    side = [inp[x] for x in ("q_I", "q_scale", "w", "k_I", "k_scale")]
    assert dsa.workspace_size(dsa.OP_FORWARD_KV4, 1, 700, 4200, wl.k, 128, 512) > \
        dsa.workspace_size(dsa.OP_FORWARD, 1, 700, 4200, wl.k, 128, 512) + 4200 * 576 * 2
    got = dsa.forward_kv4(*side, inp["q"], *cache, wl.k, wl.scale, wl.q_offset)
    low = dsa.forward_kv4(*side, inp["q"], *cache, wl.k, wl.scale, wl.q_offset, low_memory=True)
    assert all(torch.equal(a, b) for a, b in zip(got, low))
    _check(inp["q"], cache, got[0], wl.Dv, got[1], got[2], [0, 350, 699])


# the last three: every position is selected, with the keys of few rows split and of many not
@pytest.mark.parametrize("B,Lq,Lk,off", [(2, 1500, 6000, 900), (1, 700, 20000, 1400), (3, 40, 9000, 2100),
                                         (3, 1, 2500, 1499), (1, 4, 3000, 2044), (2, 300, 3000, 70)])
def test_forward_at_the_start_of_a_longer_cache(B, Lq, Lk, off):
    # the rows behind q_offset + Lq - 1 hold nothing yet: none of them may count or be read
    wl = WORKLOADS["prefill_8k"].with_(B=B, Lq=Lq, Lk=Lk, q_offset=off)
    inp = make_inputs(wl, DEV, 1)
    end = off + Lq
    cache = _cache(inp["kv"], wl.Dv)
    side = [inp[x] for x in ("q_I", "q_scale", "w", "k_I", "k_scale")]
    short = side[:3] + [side[3][:, :end].contiguous(), side[4][:, :end].contiguous()]
    want = dsa.forward_kv4(*short, inp["q"], *(t[:, :end].contiguous() for t in cache), wl.k, wl.scale, off)
    cache[1][:, end:] = float("nan")
    cache[2][:, end:] = float("nan")
    for low in (False, True):
        got = dsa.forward_kv4(*side, inp["q"], *cache, wl.k, wl.scale, off, low_memory=low)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    _check(inp["q"], cache, got[0], wl.Dv, got[1], got[2], [0, B * Lq // 2, B * Lq - 1])


@pytest.mark.parametrize("shape", ["mla", "tiny"])
@pytest.mark.parametrize("B,Lq,Lk,k", [(1, 4, 3, 2048), (2, 9, 1, 700)])
def test_more_queries_than_cache_rows(shape, B, Lq, Lk, k):
    q, kv, d_v, g = _inputs(shape, B, Lq, Lk, 21)
    cache = _cache(kv, d_v)
    idx = _indices(g, B, Lq, Lk, k, "holes")
    need = dsa.workspace_size(dsa.OP_SPARSE_ATTN, B, Lq, Lk, k, q.shape[2], d_v)
    assert need > 0
    out, lse = dsa.sparse_attn_kv4(q, *cache, idx, SCALE, workspace=torch.empty(need, device=DEV, dtype=torch.uint8))
    _check(q, cache, idx, d_v, out, lse)
    for o, l in (dsa.sparse_attn_kv4(q, *cache, idx, SCALE), dsa.sparse_attn(q, dsa.kv4_read(*cache, Lk), idx, d_v, SCALE)):
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_rows_behind_four_gigabytes():
    q, kv, d_v, g = _inputs("mla", 2, 1, 64, 6)
    Lk = 9_000_000                                         # 2 x 2.3 GB of codes
    cache = [torch.empty(2, Lk, n, dtype=t, device=DEV) for n, t in
             ((256, torch.uint8), (16, torch.bfloat16), (64, torch.bfloat16))]
    start = torch.full((2,), Lk - 64, device=DEV, dtype=torch.int32)
    dsa.kv4_write(kv, *cache, start=start)
    idx = (Lk - 64 + torch.arange(64, device=DEV, dtype=torch.int32)).expand(2, 1, 64).contiguous()
    out, lse = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    _check(q, cache, idx, d_v, out, lse)


@pytest.mark.parametrize("name,kw", [("prefill_8k", dict(B=1, Lq=300, Lk=2600, q_offset=2300)),
                                     ("prefill_8k", dict(B=2, Lq=333, Lk=1500, q_offset=1167)),   # every position selected
                                     ("prefill_8k", dict(B=3, Lq=1, Lk=5000, q_offset=4999)),
                                     ("tiny", dict(B=1, Lq=500, Lk=500, q_offset=0))])
def test_forward(name, kw):
    wl = WORKLOADS[name].with_(**kw)
    inp = make_inputs(wl, DEV, 1)
    cache = _cache(inp["kv"], wl.Dv)
    side = [inp[x] for x in ("q_I", "q_scale", "w", "k_I", "k_scale")]
    idx, out, lse = dsa.forward_kv4(*side, inp["q"], *cache, wl.k, wl.scale, wl.q_offset)
    want, _, _ = dsa.forward(*side, inp["q"], inp["kv"], wl.k, wl.Dv, wl.scale, wl.q_offset)
    assert torch.equal(idx, want)                          # the selection does not read the latent rows
    o2, l2 = dsa.sparse_attn_kv4(inp["q"], *cache, idx, wl.scale)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    sel = torch.empty(wl.B, wl.Lq, wl.k, device=DEV)
    low = dsa.forward_kv4(*side, inp["q"], *cache, wl.k, wl.scale, wl.q_offset, sel_scores=sel, low_memory=True)
    assert all(torch.equal(a, b) for a, b in zip(low, (idx, out, lse)))
    _check(inp["q"], cache, idx, wl.Dv, out, lse, [0, wl.B * wl.Lq // 2, wl.B * wl.Lq - 1])


def test_the_operators_as_a_layer_uses_them():
    """A prompt and then single tokens through norm and rotation, the 4-bit cache and both
    attentions, against the 64-bit forms of the same steps on what each step was given."""
    B, L, H, D, d_v = 2, 150, 128, 576, 512
    g = torch.Generator(device=DEV).manual_seed(11)
    inv = (10000.0 ** (-torch.arange(32, device=DEV) / 32)).float()
    w = 1 + 0.1 * torch.randn(512, generator=g, device=DEV)
    cache = dsa.kv4_cache(B, 200, D, d_v)
    start = torch.tensor([0, 30], device=DEV, dtype=torch.int32)
    latent = dict(norm="rms", weight=w, norm_dim=512, rot_start=512, interleaved=True)
    for step, n in enumerate((L, 1, 1)):
        x = torch.randn(B, n, 1, D, generator=g, device=DEV, dtype=torch.bfloat16)
        qx = torch.randn(B, n, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
        pos = (start[:, None] + torch.arange(n, device=DEV, dtype=torch.int32)).contiguous()
        rows = dsa.norm_rope(x, inv, positions=pos, **latent).squeeze(2)
        q = dsa.norm_rope(qx, inv, positions=pos, rot_start=512, interleaved=True)
        dsa.kv4_write(rows, *cache, start=start)
        held = dsa.kv4_read(*cache, n, start=start)
        assert torch.equal(held.double(), R.kv4_quantised(rows, d_v)[0])
        idx = torch.where(torch.arange(200, device=DEV) <= pos[..., None], torch.arange(200, device=DEV), -1).int()
        out, lse = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
        _check(q, cache, idx, d_v, out, lse, [0, B * n - 1])
        # a window as wide as the sequence sees the same keys
        o2, l2 = dsa.window_attn(q, dsa.kv4_read(*cache, 200), d_v, SCALE, 200, start=start)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        start += n


def test_streams_graphs_and_two_calls_at_once():
    q, kv, d_v, g = _inputs("mla", 4, 1, 3000, 9)
    cache = _cache(kv, d_v)
    idx = _indices(g, 4, 1, 3000, 2048, "prefix")
    want = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    q2 = q.neg()
    want2 = dsa.sparse_attn_kv4(q2, *cache, idx, SCALE)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [dsa.sparse_attn_kv4(q if i % 2 == 0 else q2, *cache, idx, SCALE, stream=s1 if i % 2 == 0 else s2) for i in range(6)]
    s1.synchronize()
    s2.synchronize()
    for i, (o, l) in enumerate(got):
        wo, wl = want if i % 2 == 0 else want2
        assert torch.equal(o, wo) and torch.equal(l, wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want2[0]) and torch.equal(l, want2[1])


def test_binding_refuses():
    q, kv, d_v, g = _inputs("mla", 1, 2, 8, 1)
    cache = _cache(kv, d_v)
    idx = torch.zeros(1, 2, 4, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        dsa.sparse_attn_kv4(q[..., :500].contiguous(), *cache, idx, SCALE)
    with pytest.raises(TypeError):
        dsa.sparse_attn_kv4(q, *cache, idx.long(), SCALE)
    with pytest.raises(ValueError):
        dsa.sparse_attn_kv4(q, *cache, idx[:, :1], SCALE)
    with pytest.raises(ValueError):
        dsa.sparse_attn_kv4(q, cache[0], cache[1][..., :8].contiguous(), cache[2], idx, SCALE)
    with pytest.raises(dsa.DSAError):
        dsa.sparse_attn_kv4(q, *cache, torch.zeros(1, 2, 2049, dtype=torch.int32, device=DEV), SCALE)
    with pytest.raises(dsa.DSAError):
        dsa.sparse_attn_kv4(q, *cache, idx, -1.0)
