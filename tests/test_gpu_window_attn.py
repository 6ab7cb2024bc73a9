"""Sliding window and sinks against the 64-bit form over the definition of what a query
sees, and bit for bit against dsa_sparse_attn over the same keys as an index list."""
import math

import pytest
import torch

import ref_ops as R
import sparse_attention_19_b200 as dsa

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


def _inputs(shape, B, Lq, Lk, seed):
    H, D, d_v = SHAPES[shape]
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(B, Lq, H, D, generator=g, device=DEV, dtype=torch.bfloat16),
            torch.randn(B, Lk, D, generator=g, device=DEV, dtype=torch.bfloat16), d_v)


def _seen(Lk, t, window, sinks):
    s = torch.arange(Lk, device=DEV)
    return (s <= t) & ((s > t - window) | (s < sinks))


def _check(q, kv, d_v, t_of, window, sinks, out, lse, rows):
    B, Lq, H, D = q.shape
    Lk = kv.shape[1]
    for n in rows:
        b, i = divmod(n, Lq)
        t = t_of(b) + i
        keys = _seen(Lk, t, window, sinks).nonzero().squeeze(-1)
        o, l = out[b, i].double()[None], lse[b, i].double()[None]
        if keys.numel() == 0:
            assert (o == 0).all() and (l == -math.inf).all()
            continue
        kr, valid = kv[b, keys][None], torch.ones(1, keys.numel(), dtype=torch.bool, device=DEV)
        ro, rl, p = R.attention(q[b, i][None], kr, valid, d_v, SCALE)
        to, tl = R.attention_tolerance(q[b, i][None], kr, valid, ro, rl, p, d_v, SCALE)
        assert ((o - ro).abs() <= to).all(), (n, ((o - ro).abs() / to).max())
        assert ((l - rl).abs() <= tl).all()


def _rows(B, Lq):
    n = B * Lq
    return sorted({0, 1 % n, n // 2, n - 1, n // 3, (7 * n) // 9, (Lq - 1) % n, Lq % n, 74 % n})


@pytest.mark.parametrize("shape", ["mla", "tiny"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (64, 0), (127, 1), (128, 4), (129, 16), (200, 130), (512, 16),
                                          (700, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_prefill(shape, window, sinks):
    for B, Lq, Lk, off in ((1, 333, 333, 0), (2, 85, 600, 515)):
        q, kv, d_v = _inputs(shape, B, Lq, Lk, window % 1000 + sinks % 1000)
        out, lse = dsa.window_attn(q, kv, d_v, SCALE, window, sinks, q_offset=off)
        _check(q, kv, d_v, lambda b: off, window, sinks, out, lse, _rows(B, Lq))


@pytest.mark.parametrize("shape", ["mla", "tiny"])
@pytest.mark.parametrize("window,sinks,Lk", [(1, 0, 1), (100, 0, 700), (1024, 4, 2000), (130, 130, 1500), (1500, 16, 5000),
                                             (20000, 4, 9000), (9000, 0, 30000)])
def test_single_tokens_of_sequences_of_different_lengths(shape, window, sinks, Lk):
    for B in (1, 7, 80):
        q, kv, d_v = _inputs(shape, B, 1, Lk, B + window)
        start = torch.randint(0, Lk, (B,), device=DEV, dtype=torch.int32)
        start[0] = Lk - 1
        start[-1] = 0 if B > 1 else Lk - 1
        out, lse = dsa.window_attn(q, kv, d_v, SCALE, window, sinks, start=start)
        first = start.tolist()
        _check(q, kv, d_v, lambda b: first[b], window, sinks, out, lse, sorted({0, B // 2, B - 1}))


@pytest.mark.parametrize("window,sinks", [(96, 4), (128, 0), (300, 17), (7, 40)])
@pytest.mark.parametrize("B,Lq", [(1, 200), (3, 1)])
def test_same_bits_as_the_index_list(window, sinks, B, Lq):
    Lk = 700
    q, kv, d_v = _inputs("mla", B, Lq, Lk, 4)
    off = Lk - Lq - 3
    idx = torch.full((B, Lq, window + sinks), -1, dtype=torch.int32, device=DEV)
    for i in range(Lq):
        keys = _seen(Lk, off + i, window, sinks).nonzero().squeeze(-1)
        idx[:, i, :keys.numel()] = keys.int()
    want = dsa.sparse_attn(q, kv, idx, d_v, SCALE)
    got = dsa.window_attn(q, kv, d_v, SCALE, window, sinks, q_offset=off)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_positions_outside_the_sequence():
    B, Lk = 6, 300
    q, kv, d_v = _inputs("mla", B, 4, Lk, 2)
    start = torch.tensor([-2, Lk - 2, Lk + 50, -5, 2147483647, -2147483648], device=DEV, dtype=torch.int32)
    first = start.tolist()
    for window, sinks in ((40, 3), (52, 0), (400, 0), (1, 0), (2 ** 31 - 1, 0)):
        out, lse = dsa.window_attn(q, kv, d_v, SCALE, window, sinks, start=start)
        _check(q, kv, d_v, lambda b: first[b], window, sinks, out, lse, range(B * 4))


@pytest.mark.parametrize("Lq,start,window,sinks", [(1, 400, 100, 4), (3, 200, 128, 0), (1, 900, 700, 20), (2, 5, 50, 3),
                                                   (100, 300, 64, 0)])
def test_keys_that_no_query_sees_may_hold_anything(Lq, start, window, sinks):
    q, kv, d_v = _inputs("mla", 2, Lq, 1024, 8)
    first = torch.tensor([start, start + 7], device=DEV, dtype=torch.int32)
    want = dsa.window_attn(q, kv, d_v, SCALE, window, sinks, start=first)
    for b in range(2):
        any_ = torch.zeros(1024, dtype=torch.bool, device=DEV)
        for i in range(Lq):
            any_ |= _seen(1024, start + 7 * b + i, window, sinks)
        kv[b, ~any_] = float("nan")
    got = dsa.window_attn(q, kv, d_v, SCALE, window, sinks, start=first)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(got[0].float()).all()


def test_a_window_over_everything_is_dense_causal_attention():
    q, kv, d_v = _inputs("mla", 1, 260, 260, 3)
    out, lse = dsa.window_attn(q, kv, d_v, SCALE, 260)
    idx = torch.where(torch.arange(260, device=DEV) <= torch.arange(260, device=DEV)[:, None], torch.arange(260, device=DEV), -1)
    want = dsa.sparse_attn(q, kv, idx.int()[None].contiguous(), d_v, SCALE)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_streams_graphs_and_outputs_given():
    q, kv, d_v = _inputs("mla", 3, 1, 4000, 5)
    start = torch.tensor([3999, 100, 2500], device=DEV, dtype=torch.int32)
    want = dsa.window_attn(q, kv, d_v, SCALE, 1500, 4, start=start)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = dsa.window_attn(q, kv, d_v, SCALE, 1500, 4, start=start, stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    need = dsa.workspace_size(dsa.OP_WINDOW_ATTN, 3, 1, 4000, 1504, 128, 512)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.window_attn(q, kv, d_v, SCALE, 1500, 4, start=start, out=out, lse=lse, workspace=ws)
    start.copy_(torch.tensor([7, 3000, -1], device=DEV, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want = dsa.window_attn(q, kv, d_v, SCALE, 1500, 4, start=start)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and (out[2] == 0).all()
    with pytest.raises(dsa.DSAError):
        dsa.window_attn(q, kv, d_v, SCALE, 1500, 4, start=start, workspace=ws[:need - 16])
    none, l = dsa.window_attn(q, kv, d_v, SCALE, 1500, 4, start=start, want_lse=False)
    assert l is None and torch.equal(none, out)
