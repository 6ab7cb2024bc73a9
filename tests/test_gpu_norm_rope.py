"""norm_rope and its gradient against the 64-bit forms.

Tolerances.  fp32 arithmetic: a row's sums pass at most 64 roundings (32 columns of one
lane, 5 exchange steps, the formula's own), the angle is off by at most 2^-21 (its
reduced part in fp32, up to pi), so a rotated value is off by less than
64 * 2^-24 + 2 * 2^-21 < 2^-17 of the row's largest |z|.  Then one rounding to the
output type: 2^-8 of the value in bf16; in e4m3 2^-4 of it, or half the smallest step,
2^-10 of the scale."""
import pytest
import torch

import ref_ops as R
import sparse_attention_19_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (H, D, norm_dim, rot_start, F): the indexer's queries and keys, attention queries, latent
# rows, the tiny shape, a width per row split (8 to 1024 columns), heads that fill a block more than once
WIDTHS = [(64, 128, 128, 0, 32), (1, 128, 128, 0, 32), (128, 192, 128, 128, 32), (1, 576, 512, 512, 32),
          (4, 64, 64, 0, 32), (3, 8, 8, 0, 0), (2, 24, 16, 8, 8), (5, 72, 72, 8, 32), (7, 136, 64, 0, 64), (2, 256, 256, 128, 64),
          (3, 264, 256, 256, 0), (2, 512, 512, 0, 256), (1, 768, 512, 704, 32), (2, 1024, 1024, 0, 512), (130, 16, 16, 0, 8)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()


def _case(B, L, H, D, nd, F, kind, seed, wdtype=torch.float32, first=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(B, L, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    how = dict(norm=kind)
    if kind is not None:
        how["norm_dim"] = nd
        how["weight"] = (1 + 0.2 * torch.randn(nd, generator=g, device=DEV)).to(wdtype)
        if kind == "layer":
            how["bias"] = (0.2 * torch.randn(nd, generator=g, device=DEV)).to(wdtype)
    inv = (10000.0 ** (-torch.arange(F, device=DEV, dtype=torch.float64) / max(F, 1))).float() if F else None
    pos = (first + torch.randint(0, 1000, (B, 1), generator=g, device=DEV, dtype=torch.int64)
           + torch.arange(L, device=DEV)).to(torch.int32)
    return x, inv, pos, how


def _ref_args(how):
    return dict(weight=how.get("weight"), bias=how.get("bias"), kind=how["norm"], norm_dim=how.get("norm_dim", 0))


def _check(got, y, z, e4m3):
    size = z.abs().amax(-1, keepdim=True)
    if not e4m3:
        tol = 2.0 ** -8 * y.abs() + 2.0 ** -17 * size
        assert ((got.double() - y).abs() <= tol).all()
        return
    codes, scale = got
    want = y.abs().amax((-2, -1)).clamp_min(1e-30) / 448.0
    assert ((scale.double() - want).abs() <= 2.0 ** -16 * want).all()
    s = scale.double()[..., None, None]
    off = (codes.float().double() * s - y).abs()
    assert (off <= 2.0 ** -4 * y.abs() + (2.0 ** -10 + 2.0 ** -15 * 448) * s).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kind", ["rms", "layer", None])
@pytest.mark.parametrize("H,D,nd,rs,F", WIDTHS)
def test_forward(H, D, nd, rs, F, kind, e4m3):
    for interleaved, B, L in ((False, 2, 5), (True, 1, 1), (False, 1, 67)):
        x, inv, pos, how = _case(B, L, H, D, nd, F, kind, H * D + L)
        got = dsa.norm_rope(x, inv, rot_start=rs, interleaved=interleaved, positions=pos, e4m3=e4m3, **how)
        y, z = R.norm_rope(x, pos, inv, rot_start=rs, interleaved=interleaved, **_ref_args(how))
        _check(got, y, z, e4m3)


@pytest.mark.parametrize("kind", ["rms", "layer", None])
@pytest.mark.parametrize("H,D,nd,rs,F", WIDTHS)
def test_gradient(H, D, nd, rs, F, kind):
    for interleaved, B, L in ((False, 2, 5), (True, 1, 1), (False, 1, 131)):
        x, inv, pos, how = _case(B, L, H, D, nd, F, kind, H * D + L + 1)
        dy = torch.randn_like(x)
        dx, dw, db = dsa.norm_rope_bwd(dy, x, inv, rot_start=rs, interleaved=interleaved, positions=pos, **how)
        rx, rw, rb, size = R.norm_rope_bwd(dy, x, pos, inv, rot_start=rs, interleaved=interleaved, **_ref_args(how))
        dzmax = dy.double().abs().amax(-1, keepdim=True) * 2
        # 64 roundings of the row's sums, and the angle's 2^-20 of |dz| times r |w| (in size already)
        tol = 2.0 ** -8 * rx.abs() + (64 * 2.0 ** -24 + 2.0 ** -20) * size["dx"] + 2.0 ** -17 * dzmax
        assert ((dx.double() - rx).abs() <= tol).all()
        # the sums over the rows: at most rows + 200 additions deep, every term off by
        # 64 * 2^-24 of itself and by the angle's error times |dz| of its pair
        if kind is not None:
            n = B * L * H
            xhat_size = (x.double()[..., :nd].abs().amax() * 4)
            slack = 2.0 ** -19 * n * dzmax.max() * xhat_size * 2.0 ** -2
            assert ((dw.double() - rw).abs() <= (n + 300) * 2.0 ** -24 * size["dw"] + slack).all()
            if kind == "layer":
                assert ((db.double() - rb).abs() <= (n + 300) * 2.0 ** -24 * size["db"] + slack).all()
            else:
                assert db is None


def test_gradient_against_differences():
    # the directional derivative of the 64-bit form, against the kernel's gradients
    x, inv, pos, how = _case(2, 9, 4, 64, 64, 16, "layer", 3)
    dy, v = torch.randn_like(x), torch.randn_like(x).double()
    wv, bv = torch.randn(64, device=DEV).double(), torch.randn(64, device=DEV).double()
    dx, dw, db = dsa.norm_rope_bwd(dy, x, inv, positions=pos, **how)

    def f(h):
        y, _ = R.norm_rope(x.double() + h * v, pos, inv, weight=how["weight"].double() + h * wv,
                           bias=how["bias"].double() + h * bv, kind="layer", norm_dim=64)
        return (y * dy.double()).sum()

    h = 1e-5
    diff = (f(h) - f(-h)) / (2 * h)
    got = (dx.double() * v).sum() + (dw.double() * wv).sum() + (db.double() * bv).sum()
    # every dx is rounded to bf16 once
    assert abs(diff - got) <= 2.0 ** -8 * (dx.double().abs() * v.abs()).sum() * 1.01 + 1e-3


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
def test_strided_slices_and_weight_types(wdtype):
    # heads 2..5 of a fused buffer with other columns around them
    g = torch.Generator(device=DEV).manual_seed(9)
    buf = torch.randn(2, 7, 9, 160, generator=g, device=DEV, dtype=torch.bfloat16)
    x = buf[:, :, 2:6, 16:144]
    _, inv, pos, how = _case(2, 7, 4, 128, 128, 32, "rms", 9, wdtype)
    got = dsa.norm_rope(x, inv, positions=pos, **how)
    y, z = R.norm_rope(x, pos, inv, **_ref_args(how))
    _check(got, y, z, False)
    assert torch.equal(got, dsa.norm_rope(x.contiguous(), inv, positions=pos, **how))
    # heads before tokens in memory, and one row read by every head
    t = buf.permute(0, 2, 1, 3)[..., :128]
    assert torch.equal(dsa.norm_rope(t, inv, positions=torch.arange(18, device=DEV, dtype=torch.int32).view(2, 9), **how),
                       dsa.norm_rope(t.contiguous(), inv, positions=torch.arange(18, device=DEV, dtype=torch.int32).view(2, 9), **how))
    one = x[:, :, :1].expand(-1, -1, 4, -1)
    assert torch.equal(dsa.norm_rope(one, inv, positions=pos, **how),
                       dsa.norm_rope(one.contiguous(), inv, positions=pos, **how))
    dy = torch.randn(2, 7, 4, 128, device=DEV, dtype=torch.bfloat16)
    for a, b in zip(dsa.norm_rope_bwd(dy, one, inv, positions=pos, **how),
                    dsa.norm_rope_bwd(dy, one.contiguous(), inv, positions=pos, **how)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_far_positions_and_the_default_ones():
    far = 2 ** 31 - 2000
    x, inv, pos, how = _case(2, 33, 2, 64, 64, 32, "rms", 4, first=far)
    y, z = R.norm_rope(x, pos, inv, **_ref_args(how))
    _check(dsa.norm_rope(x, inv, positions=pos, **how), y, z, False)
    want = torch.arange(17, 50, device=DEV, dtype=torch.int32).expand(2, 33).contiguous()
    assert torch.equal(dsa.norm_rope(x, inv, q_offset=17, **how), dsa.norm_rope(x, inv, positions=want, **how))


def test_zero_rows_and_values_that_are_not_finite():
    x, inv, pos, how = _case(1, 4, 2, 64, 64, 32, None, 6)
    x[0, 1] = 0
    x[0, 2, 1, 5] = float("nan")
    x[0, 3, 0, 40] = float("inf")
    codes, scale = dsa.norm_rope(x, None, e4m3=True, **how)
    assert abs(scale[0, 1].item() * 448.0 / 1e-30 - 1) < 2.0 ** -21 and (codes[0, 1].float() == 0).all()
    assert scale[0, 2].isnan() and scale[0, 3].isinf()
    clean, cscale = dsa.norm_rope(x[:, :1], None, e4m3=True, **how)
    assert torch.equal(codes[:, :1].view(torch.uint8), clean.view(torch.uint8)) and torch.equal(scale[:, :1], cscale)
    y = dsa.norm_rope(x, inv, positions=pos, norm="rms", weight=torch.ones(64, device=DEV))
    assert torch.isfinite(y[0, :2].float()).all()                  # an all-zero row stays zero (eps > 0)
    assert (y[0, 1] == 0).all() and torch.isfinite(y[0, 2, 0].float()).all()   # other heads are not touched


def test_same_bits_again_on_another_stream_and_from_a_graph():
    x, inv, pos, how = _case(3, 700, 8, 128, 128, 32, "layer", 8)
    dy = torch.randn_like(x)
    first = dsa.norm_rope_bwd(dy, x, inv, positions=pos, **how)
    y = dsa.norm_rope(x, inv, positions=pos, e4m3=True, **how)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    again = dsa.norm_rope_bwd(dy, x, inv, positions=pos, stream=st, **how)
    y2 = dsa.norm_rope(x, inv, positions=pos, e4m3=True, stream=st, **how)
    st.synchronize()
    for a, b in zip(list(first) + list(y), list(again) + list(y2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1 = dsa.norm_rope_bwd(dy, x, inv, positions=pos, **how)
        g2 = dsa.norm_rope(x, inv, positions=pos, e4m3=True, **how)
    x.neg_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    now = list(dsa.norm_rope_bwd(dy, x, inv, positions=pos, **how)) + list(dsa.norm_rope(x, inv, positions=pos, e4m3=True, **how))
    for a, b in zip(list(g1) + list(g2), now):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_the_indexer_takes_the_e4m3_output():
    g = torch.Generator(device=DEV).manual_seed(2)
    B, L, H, D = 1, 96, 64, 128
    q, k = (torch.randn(B, L, h, D, generator=g, device=DEV, dtype=torch.bfloat16) for h in (H, 1))
    w = torch.randn(B, L, H, generator=g, device=DEV, dtype=torch.bfloat16)
    inv = (10000.0 ** (-torch.arange(32, device=DEV) / 32)).float()
    qc, qs = dsa.norm_rope(q, inv, norm="rms", weight=torch.ones(D, device=DEV), e4m3=True)
    kc, ks = dsa.norm_rope(k, inv, norm="layer", weight=torch.ones(D, device=DEV), e4m3=True)
    got = dsa.indexer_scores(qc, qs, w, kc.squeeze(2), ks)
    qv, kv = qc.double() * qs.double()[..., None, None], kc.squeeze(2).double() * ks.double()[..., None]
    x = torch.einsum("blhd,bsd->blhs", qv, kv).relu()
    want = torch.einsum("blh,blhs->bls", w.double(), x)
    size = torch.einsum("blh,blhs->bls", w.double().abs(), x)
    seen = torch.ones(L, L, device=DEV, dtype=torch.bool).tril()
    # exact products, fp32 sums: 128 per product and 64 heads, every term off by < 2^-16 of its size
    assert ((got.double() - want).abs()[0][seen] <= 2.0 ** -15 * size[0][seen] + 1e-6).all()
