"""norm_rope and its gradient with so many rows that a block takes several steps, several
spans of tokens, or both, a last step and span that are not full among them: every row against
the 64-bit forms, with the tolerances of the shorter cases."""
import pytest
import torch

import ref_ops as R
import sparse_attention_19_b200 as dsa
from test_gpu_norm_rope import _case, _check, _ref_args

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (B, L, H, D, norm_dim, rot_start, F, interleaved) and what blocks do on 148 SMs
MANY = [(3, 701, 64, 128, 128, 0, 32, False),        # 4 to 8 steps a span, one short span
        (1, 5003, 64, 128, 128, 0, 32, True),        # 9 to 17 steps a span
        (1, 70001, 1, 128, 128, 0, 32, False),       # 2 to 4 spans a block, 49 tokens in the last
        (1, 3001, 2, 1024, 1024, 0, 512, False),     # 3 to 6 spans a block, a widest angle table
        (1, 9001, 1, 576, 512, 512, 32, True),       # latent rows: 2 to 4 steps a span
        (1, 1501, 128, 192, 128, 128, 32, True),     # a token's heads in two steps, 4 to 6 tokens a span
        (2, 4099, 5, 72, 72, 8, 32, False),          # heads that leave groups of lanes without a row
        (1, 160001, 16, 16, 16, 0, 8, False),        # 64 steps a span and 2 to 3 spans a block
        (1, 40009, 3, 8, 8, 0, 0, False),            # no rotation
        (1, 4099, 16, 192, 192, 64, 64, False)]      # half the row rotated


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("B,L,H,D,nd,rs,F,inter", MANY)
def test_forward(B, L, H, D, nd, rs, F, inter, kind, e4m3):
    x, inv, pos, how = _case(B, L, H, D, nd, F, kind, H * D + L)
    got = dsa.norm_rope(x, inv, rot_start=rs, interleaved=inter, positions=pos, e4m3=e4m3, **how)
    y, z = R.norm_rope(x, pos, inv, rot_start=rs, interleaved=inter, **_ref_args(how))
    _check(got, y, z, e4m3)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("B,L,H,D,nd,rs,F,inter", MANY)
def test_gradient_of_the_rows(B, L, H, D, nd, rs, F, inter, kind):
    x, inv, pos, how = _case(B, L, H, D, nd, F, kind, H * D + L + 1)
    dy = torch.randn_like(x)
    dx, dw, db = dsa.norm_rope_bwd(dy, x, inv, rot_start=rs, interleaved=inter, positions=pos, **how)
    rx, rw, rb, size = R.norm_rope_bwd(dy, x, pos, inv, rot_start=rs, interleaved=inter, **_ref_args(how))
    dzmax = dy.double().abs().amax(-1, keepdim=True) * 2
    tol = 2.0 ** -8 * rx.abs() + (64 * 2.0 ** -24 + 2.0 ** -20) * size["dx"] + 2.0 ** -17 * dzmax
    assert ((dx.double() - rx).abs() <= tol).all()
    # Sums over the rows.  A term dz xhat is off by 2^-20 of the pair's |dy| (angle and
    # rotation) times |xhat|, by 64 * 2^-24 of itself (the norm), and for the layer norm by the
    # mean's error, 64 * 2^-24 of the row's mean |x| times r, below 2^-18, times |dz|; the sums
    # are at most 400 additions deep, each 2^-24 of what is added up.
    n = B * L * H
    rough = dzmax.mean() * n                               # sum over the rows of a bound of |dz| 2
    far = 2.0 ** -20 * 4 * rough + 2.0 ** -18 * rough + 400 * 2.0 ** -24 * size["dw"]
    assert ((dw.double() - rw).abs() <= 64 * 2.0 ** -24 * size["dw"] + far).all()
    if kind == "layer":
        assert ((db.double() - rb).abs() <= 2.0 ** -20 * rough + 400 * 2.0 ** -24 * size["db"]).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("B,L,H,D,nd,rs,F,inter", MANY)
def test_gradient_sums_take_every_row_once(B, L, H, D, nd, rs, F, inter, kind):
    """Rows of +-1 with mean 0 (eps = 0: 1/std is 1), positions 0 and dy = +-1: every term of dw and
    db is +-1 and their sums, below 2^24, are exact.  A row too few or too many shifts them by 1."""
    g = torch.Generator(device=DEV).manual_seed(L)
    sign = torch.randint(0, 2, (B, L, H, 1), generator=g, device=DEV) * 2 - 1
    alternate = 1 - 2 * (torch.arange(D, device=DEV) % 2)
    x = (sign * alternate).bfloat16()
    dy = (torch.randint(0, 2, (B, L, H, D), generator=g, device=DEV, dtype=torch.int8) * 2 - 1).bfloat16()
    pos = torch.zeros(B, L, device=DEV, dtype=torch.int32)
    inv = torch.ones(F, device=DEV) if F else None
    bias = torch.zeros(nd, device=DEV) if kind == "layer" else None
    _, dw, db = dsa.norm_rope_bwd(dy, x, inv, weight=torch.ones(nd, device=DEV), bias=bias, norm=kind, norm_dim=nd,
                                  eps=0.0, rot_start=rs, interleaved=inter, positions=pos)
    assert torch.equal(dw.double(), (dy.double() * x.double())[..., :nd].sum((0, 1, 2)))
    if kind == "layer":
        assert torch.equal(db.double(), dy.double()[..., :nd].sum((0, 1, 2)))


def test_rows_behind_four_gigabytes():
    # 2.3e9 elements: byte and element offsets pass 32 bits in x, dy and every output
    B, L, H, D = 2, 35500, 64, 512
    g = torch.Generator(device=DEV).manual_seed(1)
    row = torch.randn(B, 500, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    dy_row = torch.randn(B, 500, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    x, dy = (torch.empty(B, L, H, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    for i in range(0, L, 500):
        x[:, i:i + 500], dy[:, i:i + 500] = row, dy_row
    inv = (10000.0 ** (-torch.arange(64, device=DEV) / 64)).float()
    w = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    pos = (torch.arange(L, device=DEV, dtype=torch.int32) % 500).expand(B, L).contiguous()   # every 500 rows again
    how = dict(norm="rms", weight=w, rot_start=384)
    y = dsa.norm_rope(x, inv, positions=pos, **how)
    want = dsa.norm_rope(row, inv, positions=pos[:, :500].contiguous(), **how)
    assert all(torch.equal(y[:, i:i + 500], want) for i in range(0, L, 500))
    del y
    codes, scale = dsa.norm_rope(x, inv, positions=pos, e4m3=True, **how)
    wc, ws = dsa.norm_rope(row, inv, positions=pos[:, :500].contiguous(), e4m3=True, **how)
    assert all(torch.equal(codes[:, i:i + 500].view(torch.uint8), wc.view(torch.uint8)) for i in range(0, L, 500))
    assert all(torch.equal(scale[:, i:i + 500], ws) for i in range(0, L, 500))
    del codes
    dx, dw, _ = dsa.norm_rope_bwd(dy, x, inv, positions=pos, **how)
    wx, ww, _ = dsa.norm_rope_bwd(dy_row, row, inv, positions=pos[:, :500].contiguous(), **how)
    assert all(torch.equal(dx[:, i:i + 500], wx) for i in range(0, L, 500))
    # 71 times the sums of one part: 4.5e6 terms of about 1, each sum at most 600 additions deep
    size = (dy_row.double().abs().amax() * row.double().abs().amax() * 2)
    assert ((dw.double() - 71 * ww.double()).abs() <= 1200 * 2.0 ** -24 * size * B * L * H).all()
