"""The 4-bit latent cache: what is stored and read back equals the 64-bit form bit for bit
(every step of the definition is exact in fp32: see the CPU tests of the form)."""
import pytest
import torch

import ref_ops as R
import sparse_attention_19_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHAPES = [(576, 512), (192, 128)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()


def _rows(B, L, d_qk, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kv = torch.randn(B, L, d_qk, generator=g, device=DEV, dtype=torch.bfloat16)
    # magnitudes over the whole range of bf16, and values that lie halfway between two codes
    kv[:, ::3] *= torch.exp2(torch.randint(-90, 90, (B, (L + 2) // 3, 1), generator=g, device=DEV).float()).bfloat16()
    kv[:, 1::3] = (kv[:, 1::3].float() * 4).round().clamp(-14, 14).bfloat16() / 2
    return kv


def _garbage(B, Lk, d_qk, d_v):
    codes, scales, tail = dsa.kv4_cache(B, Lk, d_qk, d_v)
    codes.fill_(0x5A)
    scales.fill_(3.0)
    tail.fill_(-7.0)
    return codes, scales, tail


@pytest.mark.parametrize("d_qk,d_v", SHAPES)
@pytest.mark.parametrize("B,L,Lk", [(1, 1, 1), (3, 7, 20), (2, 129, 300), (64, 1, 33)])
def test_store_and_read_back(B, L, Lk, d_qk, d_v):
    kv = _rows(B, L, d_qk, B * L)
    start = torch.randint(0, Lk - L + 1, (B,), device=DEV, dtype=torch.int32)
    cache = _garbage(B, Lk, d_qk, d_v)
    before = [t.clone() for t in cache]
    dsa.kv4_write(kv, *cache, start=start)
    want, step = R.kv4_quantised(kv, d_v)
    got = dsa.kv4_read(*cache, L, start=start)
    assert torch.equal(got.double(), want)
    # the layout, by its own description
    at = torch.arange(B, device=DEV)[:, None]
    rows = start.long()[:, None] + torch.arange(L, device=DEV)
    assert torch.equal(R.kv4_values(*(t[at, rows] for t in cache)), want)
    # rows around them are left as they were
    touched = torch.zeros(B, Lk, dtype=torch.bool, device=DEV)
    touched[at, rows] = True
    for now, then in zip(cache, before):
        assert torch.equal(now[~touched], then[~touched])


def test_rows_outside_the_cache():
    kv = _rows(4, 5, 576, 1)
    start = torch.tensor([-3, 6, 2147483647, -2147483648], device=DEV, dtype=torch.int32)
    cache = _garbage(4, 8, 576, 512)
    before = [t.clone() for t in cache]
    dsa.kv4_write(kv, *cache, start=start)
    want, _ = R.kv4_quantised(kv, 512)
    got = dsa.kv4_read(*cache, 5, start=start)
    assert torch.equal(got[0, 3:].double(), want[0, 3:]) and (got[0, :3] == 0).all()
    assert torch.equal(got[1, :2].double(), want[1, :2]) and (got[1, 2:] == 0).all()
    assert (got[2:] == 0).all()
    for now, then in zip(cache, before):
        assert torch.equal(now[0, 2:], then[0, 2:]) and torch.equal(now[1, :6], then[1, :6])
        assert torch.equal(now[2:], then[2:])
    dsa.kv4_write(kv, *cache, offset=3)
    assert torch.equal(dsa.kv4_read(*cache, 5, offset=3).double(), want)


def test_groups_without_a_step():
    kv = _rows(1, 5, 576, 2)
    kv[0, 0, :32] = 0
    kv[0, 1, 32:64] = 2.0 ** -101
    kv[0, 2, 70] = float("nan")
    kv[0, 3, 100] = float("inf")
    kv[0, 4, 130] = 3.0e38
    kv[0, 4, 512] = float("inf")                       # the tail is held as it is
    cache = dsa.kv4_cache(1, 5, 576, 512)
    dsa.kv4_write(kv, *cache)
    got = dsa.kv4_read(*cache, 5)
    want, _ = R.kv4_quantised(kv, 512)
    assert torch.equal(torch.nan_to_num(got.double(), nan=7e77), torch.nan_to_num(want, nan=7e77))
    assert (got[0, 0, :32] == 0).all() and (got[0, 1, 32:64] == 0).all()
    assert got[0, 2, 64:96].isnan().all() and got[0, 3, 96:128].isnan().all() and got[0, 4, 128:160].isnan().all()
    assert got.isnan().sum() == 96 and got[0, 4, 512].isinf()


def test_every_pair_of_a_magnitude_and_its_group():
    # every bf16 magnitude of two octaves against a group maximum: rounding, ties and steps
    a = (torch.arange(0, 512, device=DEV) / 256.0).bfloat16()
    top = (1.0 + torch.arange(0, 128, device=DEV) / 128.0).bfloat16()
    kv = torch.zeros(1, 128 * 2, 576, device=DEV, dtype=torch.bfloat16)
    vals = a[:496].view(1, 16, 31).expand(256, 16, 31)
    kv[0, :, :512] = torch.cat((top.repeat(2)[:, None, None].expand(256, 16, 1), vals), -1).flatten(-2)
    kv[0, 128:, :512] *= -1
    kv[0, :, :512].clamp_(-1.9921875, 1.9921875)
    cache = dsa.kv4_cache(1, 256, 576, 512)
    dsa.kv4_write(kv, *cache)
    want, _ = R.kv4_quantised(kv, 512)
    assert torch.equal(dsa.kv4_read(*cache, 256).double(), want)


def test_streams_graphs_and_far_rows():
    # a cache whose byte offsets pass 32 bits: 2^24 rows of 256 code bytes
    B, Lk = 3, 6_000_000
    cache = [torch.empty(B, Lk, n, dtype=t, device=DEV) for n, t in
             ((256, torch.uint8), (16, torch.bfloat16), (64, torch.bfloat16))]
    kv = _rows(B, 4, 576, 3)
    start = torch.full((B,), Lk - 4, device=DEV, dtype=torch.int32)
    want, _ = R.kv4_quantised(kv, 512)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    dsa.kv4_write(kv, *cache, start=start, stream=st)
    got = dsa.kv4_read(*cache, 4, start=start, stream=st)
    st.synchronize()
    assert torch.equal(got.double(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.kv4_write(kv, *cache, start=start)
        out = dsa.kv4_read(*cache, 4, start=start)
    kv.mul_(2)
    start.sub_(100)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.double(), R.kv4_quantised(kv, 512)[0])
