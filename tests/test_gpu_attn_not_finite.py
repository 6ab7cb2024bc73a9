"""A NaN in a row that a query attends to reaches that query's out and lse, in every form of
the attention and however a row's keys are split, and no other query's."""
import math

import pytest
import torch

import sparse_attention_19_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(192.0)
SHAPES = {"mla": (128, 576, 512), "tiny": (16, 192, 128)}
LK = 3000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    assert dsa.device_status() == 0


def _setup(shape, Lq):
    H, D, d_v = SHAPES[shape]
    g = torch.Generator(device=DEV).manual_seed(Lq)
    q = torch.randn(1, Lq, H, D, generator=g, device=DEV, dtype=torch.bfloat16)
    kv = torch.randn(1, LK, D, generator=g, device=DEV, dtype=torch.bfloat16)
    return q, kv, d_v


def _run(form, q, kv, d_v, k):
    """Query i attends to keys LK - k - Lq + i + 1 ... LK - Lq + i."""
    Lq = q.shape[1]
    if form == "window":
        return dsa.window_attn(q, kv, d_v, SCALE, k, q_offset=LK - Lq)
    t = LK - Lq + torch.arange(Lq, device=DEV)
    idx = (t[:, None] - k + 1 + torch.arange(k, device=DEV)).int()[None].contiguous()
    if form == "bf16":
        return dsa.sparse_attn(q, kv, idx, d_v, SCALE)
    cache = dsa.kv4_cache(1, LK, kv.shape[2], d_v)
    dsa.kv4_write(kv, *cache)
    return dsa.sparse_attn_kv4(q, *cache, idx, SCALE)


# few rows: their keys are split and merged; many: one unit a row
@pytest.mark.parametrize("shape,Lq", [("mla", 2), ("tiny", 2), ("mla", 170), ("tiny", 170)])
@pytest.mark.parametrize("form", ["bf16", "kv4", "window"])
@pytest.mark.parametrize("key,col", [(LK - 300, 5), (LK - 1, 0), (LK - 700, -1)])
def test_a_nan_reaches_the_queries_that_attend_to_it(shape, Lq, form, key, col):
    q, kv, d_v = _setup(shape, Lq)
    k = 640 if Lq == 2 else 384
    H = q.shape[2]
    assert (dsa.workspace_size(dsa.OP_SPARSE_ATTN, 1, Lq, LK, k, H, d_v) > 0) == (Lq == 2)
    want = _run(form, q, kv, d_v, k)
    kv[0, key, col] = float("nan")
    out, lse = _run(form, q, kv, d_v, k)
    t = LK - Lq + torch.arange(Lq, device=DEV)
    hit = (key <= t) & (key > t - k)
    assert out[0, hit].isnan().all() and lse[0, hit].isnan().all()
    assert torch.equal(out[0, ~hit], want[0][0, ~hit]) and torch.equal(lse[0, ~hit], want[1][0, ~hit])


@pytest.mark.parametrize("shape,Lq", [("mla", 2), ("tiny", 170)])
def test_a_nan_in_one_head_of_a_query_stays_there(shape, Lq):
    q, kv, d_v = _setup(shape, Lq)
    want = _run("bf16", q, kv, d_v, 640)
    q[0, 1, 3, 7] = float("nan")
    for form in ("bf16", "window"):
        out, lse = _run(form, q, kv, d_v, 640)
        assert out[0, 1, 3].isnan().all() and lse[0, 1, 3].isnan()
        hit = torch.zeros(lse.shape, dtype=torch.bool, device=DEV)
        hit[0, 1, 3] = True
        assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])


@pytest.mark.parametrize("form", ["bf16", "kv4"])
def test_a_nan_alone_among_masked_entries(form):
    # every other split of the row is empty
    q, kv, d_v = _setup("mla", 2)
    kv[0, 9, 4] = float("nan")
    idx = torch.full((1, 2, 2048), -1, device=DEV, dtype=torch.int32)
    idx[0, 0, 3] = 9
    idx[0, 1, 3] = 8
    if form == "bf16":
        out, lse = dsa.sparse_attn(q, kv, idx, d_v, SCALE)
    else:
        cache = dsa.kv4_cache(1, LK, 576, 512)
        dsa.kv4_write(kv, *cache)
        out, lse = dsa.sparse_attn_kv4(q, *cache, idx, SCALE)
    assert out[0, 0].isnan().all() and lse[0, 0].isnan().all()
    assert torch.isfinite(out[0, 1].float()).all() and torch.isfinite(lse[0, 1]).all()
