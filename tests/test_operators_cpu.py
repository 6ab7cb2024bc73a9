"""The operators around the attention without a GPU: refusals on the host before
anything is enqueued, the 64-bit forms the GPU tests compare with (the gradient
against differences), and the 4-bit cache's layout."""
import ctypes

import pytest
import torch

import ref_ops as R
import sparse_attention_19_b200 as dsa
from sparse_attention_19_b200 import build as dsa_build


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


P = ctypes.c_void_p(16)
ODD = ctypes.c_void_p(24)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _nr(**kw):
    base = dict(B=1, L=4, H=2, D=64, stride_b=512, stride_l=128, stride_h=64, x=16, norm=1, norm_dim=64, eps=1e-6,
                weight=16, bias=None, weight_bf16=0, rot_start=0, n_freq=16, interleaved=0, inv_freq=16,
                positions=None, q_offset=0)
    base.update(kw)
    return dsa.NormRopeArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(x=24), INVALID), (dict(B=0), INVALID), (dict(L=0), INVALID), (dict(H=0), INVALID),
    (dict(D=0), INVALID), (dict(norm=3), INVALID), (dict(weight=None), INVALID), (dict(weight=24), INVALID),
    (dict(norm_dim=0), INVALID), (dict(norm_dim=72), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(bias=16), INVALID), (dict(norm=2, bias=24), INVALID),
    (dict(n_freq=-8), INVALID), (dict(rot_start=-8), INVALID), (dict(inv_freq=None), INVALID),
    (dict(inv_freq=24), INVALID), (dict(positions=24), INVALID), (dict(rot_start=40), INVALID),
    (dict(stride_l=-128), INVALID), (dict(q_offset=2 ** 31 - 4), INVALID),
    (dict(D=60), INVALID), (dict(D=60, norm_dim=56), UNSUPPORTED), (dict(D=1032), UNSUPPORTED), (dict(norm_dim=60), UNSUPPORTED),
    (dict(n_freq=12), UNSUPPORTED), (dict(rot_start=4), UNSUPPORTED), (dict(stride_h=60), UNSUPPORTED),
    (dict(B=2 ** 16, L=2 ** 15), UNSUPPORTED), (dict(B=2 ** 12, L=2 ** 12, H=2 ** 8), UNSUPPORTED),
])
def test_norm_rope_refuses(L, kw, status):
    a = _nr(**kw)
    assert L.dsa_norm_rope(ctypes.byref(a), P, None, None) == status
    assert L.dsa_norm_rope(ctypes.byref(a), P, P, None) == status
    assert L.dsa_norm_rope_bwd(ctypes.byref(a), P, P, P, P if a.bias else None, P, 1 << 30, None) == status
    assert L.dsa_norm_rope_bwd_workspace(ctypes.byref(a)) == 0


def test_norm_rope_refuses_outputs_and_workspace(L):
    a = _nr()
    assert L.dsa_norm_rope(None, P, None, None) == INVALID
    assert L.dsa_norm_rope(ctypes.byref(a), None, None, None) == INVALID
    assert L.dsa_norm_rope(ctypes.byref(a), ODD, None, None) == INVALID
    assert L.dsa_norm_rope(ctypes.byref(a), P, ODD, None) == INVALID
    need = L.dsa_norm_rope_bwd_workspace(ctypes.byref(a))
    assert need > 0 and need % (64 * 4) == 0
    layer = _nr(norm=2, bias=16)
    assert L.dsa_norm_rope_bwd_workspace(ctypes.byref(layer)) == 2 * need
    f = L.dsa_norm_rope_bwd
    assert f(ctypes.byref(a), None, P, P, None, P, need, None) == INVALID
    assert f(ctypes.byref(a), P, None, P, None, P, need, None) == INVALID
    assert f(ctypes.byref(a), P, P, None, None, P, need, None) == INVALID          # no dweight
    assert f(ctypes.byref(a), P, P, P, P, P, need, None) == INVALID                # dbias without a bias
    assert f(ctypes.byref(layer), P, P, P, None, P, 2 * need, None) == INVALID     # a bias without dbias
    assert f(ctypes.byref(a), P, P, P, None, P, need - 1, None) == WORKSPACE
    assert f(ctypes.byref(a), P, P, P, None, None, need, None) == WORKSPACE
    assert f(ctypes.byref(a), P, P, P, None, ODD, need, None) == WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(Lk=0), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(tail=None), INVALID), (dict(codes=24), INVALID), (dict(scales=24), INVALID), (dict(tail=24), INVALID),
    (dict(d_qk=512), UNSUPPORTED), (dict(d_v=256), UNSUPPORTED), (dict(B=2 ** 16, Lk=2 ** 15), UNSUPPORTED),
])
def test_kv4_refuses(L, kw, status):
    base = dict(B=2, Lk=8, d_qk=576, d_v=512, codes=16, scales=16, tail=16)
    base.update(kw)
    c = dsa.Kv4Cache(**base)
    for f in (L.dsa_kv4_write, L.dsa_kv4_read):
        assert f(ctypes.byref(c), P, 1, None, 0, None) == status


def test_kv4_refuses_rows(L):
    c = dsa.Kv4Cache(2, 8, 576, 512, 16, 16, 16)
    for f in (L.dsa_kv4_write, L.dsa_kv4_read):
        assert f(None, P, 1, None, 0, None) == INVALID
        assert f(ctypes.byref(c), None, 1, None, 0, None) == INVALID
        assert f(ctypes.byref(c), ODD, 1, None, 0, None) == INVALID
        assert f(ctypes.byref(c), P, 0, None, 0, None) == INVALID
        assert f(ctypes.byref(c), P, 1, ODD, 0, None) == INVALID
        assert f(ctypes.byref(c), P, 2 ** 30, None, 0, None) == UNSUPPORTED


def _k4(**kw):
    base = dict(H=128, d_qk=576, d_v=512, scale=0.07, q=16, codes=16, scales=16, tail=16)
    base.update(kw)
    return dsa.Kv4AttnArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(tail=None), INVALID),
    (dict(codes=24), INVALID), (dict(scales=24), INVALID), (dict(tail=24), INVALID), (dict(q=24), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(H=64), UNSUPPORTED),
    (dict(d_v=256), UNSUPPORTED),
])
def test_kv4_attention_refuses(L, kw, status):
    a = _k4(**kw)
    assert L.dsa_sparse_attn_kv4(ctypes.byref(a), 1, 1, 8, P, 8, P, None, P, 1 << 40, None) == status
    ia = dsa.IndexerArgs(1, 8, 8, 0, 64, 128, 16, None, 16, 16, None)
    assert L.dsa_forward_kv4(ctypes.byref(ia), ctypes.byref(a), 8, P, None, P, None, P, 1 << 40, None) == status


def test_kv4_attention_refuses_the_rest(L):
    a = _k4()
    f = L.dsa_sparse_attn_kv4
    assert f(None, 1, 1, 8, P, 8, P, None, P, 1 << 40, None) == INVALID
    for sizes in ((0, 1, 8), (1, 0, 8), (1, 1, 0)):
        assert f(ctypes.byref(a), *sizes, P, 8, P, None, P, 1 << 40, None) == INVALID
    assert f(ctypes.byref(a), 2 ** 16, 1, 2 ** 15, P, 8, P, None, P, 1 << 40, None) == UNSUPPORTED
    assert f(ctypes.byref(a), 1, 1, 8, None, 8, P, None, P, 1 << 40, None) == INVALID
    assert f(ctypes.byref(a), 1, 1, 8, P, 8, None, None, P, 1 << 40, None) == INVALID
    assert f(ctypes.byref(a), 1, 1, 8, P, 8, P, ODD, P, 1 << 40, None) == INVALID
    assert f(ctypes.byref(a), 1, 1, 8, P, 0, P, None, P, 1 << 40, None) == UNSUPPORTED
    assert f(ctypes.byref(a), 1, 1, 8, P, 2049, P, None, P, 1 << 40, None) == UNSUPPORTED
    need = dsa.workspace_size(dsa.OP_SPARSE_ATTN, 1, 1, 4096, 2048, 128, 512)
    assert need > 0 and f(ctypes.byref(a), 1, 1, 4096, P, 2048, P, None, P, need - 1, None) == WORKSPACE
    assert f(ctypes.byref(a), 1, 1, 4096, P, 2048, P, None, None, need, None) == WORKSPACE
    ia = dsa.IndexerArgs(1, 8, 8, 0, 64, 128, 16, None, 16, 16, None)
    assert L.dsa_forward_kv4(ctypes.byref(ia), None, 8, P, None, P, None, P, 1 << 40, None) == INVALID
    assert L.dsa_forward_kv4(None, ctypes.byref(a), 8, P, None, P, None, P, 1 << 40, None) == INVALID
    assert L.dsa_forward_kv4(ctypes.byref(ia), ctypes.byref(a), 8, P, None, P, None, P, 255, None) == WORKSPACE


def test_kv4_workspace_holds_unpacked_rows_where_lists_repeat_them():
    size = dsa.workspace_size
    for B, Lq, Lk, k in [(64, 1, 32768, 2048), (1, 100, 131072, 2048), (1, 30, 100, 100)]:      # few uses of a row
        assert size(dsa.OP_SPARSE_ATTN_KV4, B, Lq, Lk, k, 128, 512) == size(dsa.OP_SPARSE_ATTN, B, Lq, Lk, k, 128, 512)
    for B, Lq, Lk, k in [(1, 1024, 32768, 2048), (4, 800, 1000, 2048), (1, 4000, 100, 300)]:
        least = size(dsa.OP_SPARSE_ATTN, B, Lq, max(Lq, Lk), k, 128, 512)
        assert size(dsa.OP_SPARSE_ATTN_KV4, B, Lq, Lk, k, 128, 512) >= least + (B * Lk + 1) * 576 * 2
    for op in (dsa.OP_SPARSE_ATTN_KV4, dsa.OP_FORWARD_KV4):
        assert size(op, 0, 1, 8, 8, 128, 512) == size(op, 1, 1, 8, 2049, 128, 512) == size(op, 1, 1, 8, 0, 128, 512) == 0
    assert size(dsa.OP_FORWARD_KV4, 1, 1, 4096, 2048, 128, 512) == size(dsa.OP_FORWARD, 1, 1, 4096, 2048, 128, 512) > 0


@pytest.mark.parametrize("B,Lq,Lk,off", [(1, 1024, 131072, 1500), (2, 1500, 6000, 900), (4, 2000, 4000, 2000),
                                         (1, 1024, 131072, 130048)])
def test_forward_workspace_holds_the_rows_that_can_be_selected(B, Lq, Lk, off):
    ia = dsa.IndexerArgs(B, Lq, Lk, off, 64, 128, 16, None, 16, 16, None)
    plain = dsa.workspace_size_args(dsa.OP_FORWARD, ia, 2048, 128, 512)
    room = dsa.workspace_size_args(dsa.OP_FORWARD_KV4, ia, 2048, 128, 512) - plain
    assert 0 <= room - (B * (off + Lq) + 1) * 576 * 2 <= 256
    # lists of the caller's may name every row
    any_ = dsa.workspace_size_args(dsa.OP_SPARSE_ATTN_KV4, ia, 2048, 128, 512)
    assert any_ == dsa.workspace_size(dsa.OP_SPARSE_ATTN_KV4, B, Lq, Lk, 2048, 128, 512)


@pytest.mark.parametrize("Lk,below,above", [(131072, 256, 512), (32768, 64, 128), (8192, 24, 64), (4096, 24, 64)])
def test_the_unpacking_rule_lies_between_what_was_measured(Lk, below, above):
    # queries of 2048 entries for which converting in the kernel was no slower, and slower
    def room(Lq):
        return dsa.workspace_size(dsa.OP_SPARSE_ATTN_KV4, 1, Lq, Lk, 2048, 128, 512) - \
            dsa.workspace_size(dsa.OP_SPARSE_ATTN, 1, Lq, Lk, 2048, 128, 512)

    assert room(below) == 0 and room(above) >= (Lk + 1) * 576 * 2


def test_forward_workspace_counts_the_entries_that_lists_hold():
    # 600 queries from position 0: t + 1 entries each, 180300 in all, over 600 rows of 131072;
    # 20 queries from position 0: 210, too few to unpack 20 rows for, whatever k is
    for Lq, unpacks in ((600, True), (20, False)):
        ia = dsa.IndexerArgs(1, Lq, 131072, 0, 64, 128, 16, None, 16, 16, None)
        room = dsa.workspace_size_args(dsa.OP_FORWARD_KV4, ia, 2048, 128, 512) - \
            dsa.workspace_size_args(dsa.OP_FORWARD, ia, 2048, 128, 512)
        assert (room > 0) == unpacks and room <= 256 + (Lq + 1) * 576 * 2


def test_workspace_of_more_queries_than_cache_rows():
    # the lists' length decides, not the rows that they name
    for B, Lq, Lk, k in [(1, 4, 3, 2048), (2, 9, 1, 700), (1, 40, 39, 2048)]:
        need = dsa.workspace_size(dsa.OP_SPARSE_ATTN, B, Lq, Lq, k, 128, 512)
        assert dsa.workspace_size(dsa.OP_SPARSE_ATTN, B, Lq, Lk, k, 128, 512) == need
        assert (need > 0) == (Lq < 40)                     # 40 rows of 16 tiles are not split
    for k in (0, 2049):
        assert dsa.workspace_size(dsa.OP_SPARSE_ATTN, 1, 4, 3, k, 128, 512) == 0
    # these place query i at position Lk - Lq + i or later
    for op in (dsa.OP_TOPK, dsa.OP_FORWARD, dsa.OP_FORWARD_LOWMEM, dsa.OP_INDEXER_TOPK, dsa.OP_WINDOW_ATTN, dsa.OP_FORWARD_KV4):
        assert dsa.workspace_size(op, 1, 4, 3, 2048, 128, 512) == 0


def test_window_attention_refuses(L):
    good = dsa.AttnArgs(128, 576, 512, 0.07, 16, 16)
    f = L.dsa_window_attn

    def call(a=good, B=1, Lq=4, Lk=8, off=0, start=None, window=4, sinks=0, out=P, lse=None, ws=P, n=1 << 40):
        return f(None if a is None else ctypes.byref(a), B, Lq, Lk, off, start, window, sinks, out, lse, ws, n, None)

    assert call(a=None) == INVALID and call(out=None) == INVALID and call(out=ODD) == INVALID
    assert call(lse=ODD) == INVALID and call(start=ODD) == INVALID
    assert call(B=0) == INVALID and call(Lq=0) == INVALID and call(Lk=0) == INVALID
    assert call(window=0) == INVALID and call(window=-1) == INVALID and call(sinks=-1) == INVALID
    assert call(off=5) == INVALID and call(off=-1) == INVALID and call(Lq=9, start=P) == INVALID
    assert call(a=dsa.AttnArgs(128, 576, 512, 0.07, None, 16)) == INVALID
    assert call(a=dsa.AttnArgs(64, 576, 512, 0.07, 16, 16)) == UNSUPPORTED
    assert call(B=2 ** 16, Lk=2 ** 15) == UNSUPPORTED
    need = dsa.workspace_size(dsa.OP_WINDOW_ATTN, 1, 4, 4096, 1000, 128, 512)
    assert need > 0 and call(Lk=4096, window=1000, n=need - 1) == WORKSPACE
    assert call(Lk=4096, window=1000, ws=None, n=need) == WORKSPACE
    # longer windows than the index lists' 2048 entries, and never more than the keys there are
    assert dsa.workspace_size(dsa.OP_WINDOW_ATTN, 1, 1, 65536, 40000, 128, 512) > 0
    assert dsa.workspace_size(dsa.OP_WINDOW_ATTN, 1, 4, 1000, 2 ** 31 - 1, 128, 512) == \
        dsa.workspace_size(dsa.OP_WINDOW_ATTN, 1, 4, 1000, 1000, 128, 512)
    assert dsa.workspace_size(dsa.OP_WINDOW_ATTN, 1, 4096, 4096, 512, 128, 512) == 0


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.norm_rope(x)
    with pytest.raises(TypeError):
        dsa.norm_rope(x.float())
    codes, scales, tail = dsa.kv4_cache(1, 4, 576, 512, device="cpu")
    assert codes.shape == (1, 4, 256) and scales.shape == (1, 4, 16) and tail.shape == (1, 4, 64)
    assert (R.kv4_values(codes, scales, tail) == 0).all()
    with pytest.raises(ValueError):
        dsa.kv4_read(codes, scales, tail, 1)


_X = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
_Q = torch.zeros(1, 4, 2, 192, dtype=torch.bfloat16)
_KV = torch.zeros(1, 8, 192, dtype=torch.bfloat16)


@pytest.mark.parametrize("name,call", [
    ("q_offset", lambda v: dsa.norm_rope(_X, q_offset=v)),
    ("rot_start", lambda v: dsa.norm_rope(_X, rot_start=v)),
    ("norm_dim", lambda v: dsa.norm_rope(_X, norm="rms", norm_dim=v)),
    ("q_offset", lambda v: dsa.norm_rope_bwd(_X, _X, q_offset=v)),
    ("offset", lambda v: dsa.kv4_write(_KV, *dsa.kv4_cache(1, 8, 192, 128, device="cpu"), offset=v)),
    ("offset", lambda v: dsa.kv4_read(*dsa.kv4_cache(1, 8, 192, 128, device="cpu"), 4, offset=v)),
    ("L", lambda v: dsa.kv4_read(*dsa.kv4_cache(1, 8, 192, 128, device="cpu"), v)),
    ("q_offset", lambda v: dsa.window_attn(_Q, _KV, 128, 1.0, 4, q_offset=v)),
])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, -2 ** 31 - 1, -2 ** 32])
def test_binding_refuses_integers_beyond_32_bits(name, call, value):
    """The C side takes 32-bit integers; a wrapped one would name another row or position."""
    with pytest.raises(ValueError, match=f"{name}.* 32 bits"):
        call(value)


@pytest.mark.parametrize("kw", [dict(window=-2 ** 32 + 5), dict(window=4, sinks=-2 ** 32)])
def test_binding_refuses_windows_far_below_zero(kw):
    with pytest.raises(ValueError, match="32 bits"):
        dsa.window_attn(_Q, _KV, 128, 1.0, **kw)


@pytest.mark.parametrize("name", ["dweight", "dbias"])
def test_binding_refuses_gradients_of_a_norm_that_is_not_there(name):
    """They would come back as they were given."""
    with pytest.raises(ValueError, match="belong to a norm"):
        dsa.norm_rope_bwd(_X, _X, **{name: torch.zeros(64)})


@pytest.mark.parametrize("kind", ["rms", "layer", None])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_form_against_differences(kind, interleaved):
    g = torch.Generator().manual_seed(5)
    x, dy, v = (torch.randn(2, 3, 2, 32, generator=g, dtype=torch.float64) for _ in range(3))
    nd, rs = 24, 8
    w, wv = (1 + 0.3 * torch.randn(nd, generator=g, dtype=torch.float64) for _ in range(2))
    b, bv = (torch.randn(nd, generator=g, dtype=torch.float64) for _ in range(2)) if kind == "layer" else (None, None)
    pos = torch.tensor([[0, 1, 7], [100000, 100001, 3]])
    inv = torch.tensor([1.0, 0.3, 0.1, 0.03, 0.01, 0.003, 0.001, 0.0003])
    how = dict(kind=kind, norm_dim=nd, rot_start=rs, interleaved=interleaved)

    def f(h):
        bias = None if b is None else b + h * bv
        y, _ = R.norm_rope(x + h * v, pos, inv, w + h * wv, bias, **how)
        return (y * dy).sum()

    dx, dw, db, _ = R.norm_rope_bwd(dy, x, pos, inv, w, b, **how)
    want = (dx * v).sum()
    if kind is not None:
        want = want + (dw * wv).sum() + (0 if b is None else (db * bv).sum())
    # central difference: error h^2/6 f''' ~ 1e-8, rounding 1e-16/h * |f| ~ 1e-10
    h = 1e-4
    assert abs((f(h) - f(-h)) / (2 * h) - want) < 1e-5 * (1 + abs(want))


@pytest.mark.parametrize("d_v", [128, 512])
def test_kv4_layout_holds_every_column_once(d_v):
    seen = {R.kv4_nibble(d_v, c) for c in range(d_v)}
    assert seen == {(b, s) for b in range(d_v // 2) for s in (0, 4)}
    slots = {}
    for c in range(d_v):
        slots.setdefault(R.kv4_scale_slot(d_v, c), set()).add(c // 32)
    assert sorted(slots) == list(range(d_v // 32)) and all(len(g) == 1 for g in slots.values())


def test_kv4_values_are_exact_in_bf16():
    g = torch.Generator().manual_seed(1)
    kv = (torch.randn(64, 576, generator=g) * torch.logspace(-20, 20, 64)[:, None]).bfloat16()
    v, step = R.kv4_quantised(kv, 512)
    assert torch.equal(v.bfloat16().double(), v)
    assert torch.equal(step.bfloat16().double(), step)
    # nothing is clipped, and no value is off by more than half a step
    x = kv[:, :512].double().unflatten(-1, (-1, 32))
    off = (v[:, :512].unflatten(-1, (-1, 32)) - x).abs()
    assert (off <= step.unsqueeze(-1) / 2).all()
