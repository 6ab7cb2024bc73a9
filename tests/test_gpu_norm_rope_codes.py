"""The e4m3 output's scale and codes, bit for bit where the row is not changed before them:
scale = max|x| / 448 and code = rne(x / scale), both quotients in fp32."""
import pytest
import torch

import sparse_attention_19_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()


def _check(x):
    codes, scale = dsa.norm_rope(x, None, e4m3=True)
    f = x.float().cpu()
    want_scale = f.abs().amax((-2, -1)).clamp_min(1e-30) / 448.0
    assert torch.equal(scale.cpu(), want_scale)
    want = (f / want_scale[..., None, None]).to(torch.float8_e4m3fn)
    assert torch.equal(codes.cpu().float(), want.float())


# 19 heads lie in one step of a block; 130 heads take the kernel that computes a token twice
@pytest.mark.parametrize("heads", [19, 130])
@pytest.mark.parametrize("exponent", [0, -60, -99, 99])
def test_every_pair_of_significands(heads, exponent):
    """Token a: its largest magnitude has significand a; behind it every significand of the 18
    binades below, so that quotients on and beside the border of two codes are all there."""
    sig = (128 + torch.arange(128, device=DEV)).double() / 128
    x = torch.zeros(1, 128, heads, 128, device=DEV, dtype=torch.float64)
    x[0, :, 0] = sig[:, None]
    for e in range(18):
        x[0, :, heads - 1 - e] = torch.where(sig * 2.0 ** -e <= sig[:, None], sig * 2.0 ** -e, 0.0)
    x[0, :, :, 1::2] *= -1
    _check((x * 2.0 ** exponent).bfloat16())


def test_random_rows_of_many_sizes():
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(2, 999, 4, 64, generator=g, device=DEV) * 2.0 ** torch.randint(
        -30, 30, (2, 999, 1, 1), generator=g, device=DEV)
    _check((x * 2.0 ** torch.randint(-14, 1, x.shape, generator=g, device=DEV)).bfloat16())


def test_an_infinity_leaves_zeros_and_a_nan():
    x = torch.randn(1, 3, 2, 64, device=DEV).bfloat16()
    x[0, 1, 0, 9] = float("-inf")
    codes, scale = dsa.norm_rope(x, None, e4m3=True)
    assert scale[0, 1].isinf() and torch.isfinite(scale[0, ::2]).all()
    c = codes.float()
    assert c[0, 1, 0, 9].isnan() and c.isnan().sum() == 1
    c[0, 1, 0, 9] = 0
    assert (c[0, 1] == 0).all()
