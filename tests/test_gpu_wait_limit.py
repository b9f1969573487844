"""Waits that run out in tiles of few steps: the loading warp has sent all its
copies by then and has no wait of its own that could fail, and the MMA warp
may have issued its last product. The copies and products still have to end
before the CTA does, so that a call afterwards gives the bits it gave before.

The limits: one SM cycle (the first wait gives up), and some within a tile's
life, so that other waits do, the one for the accumulators among them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LIMITS = (1, 300, 1000, 2000, 3000, 5000)


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


def full_pattern(losa, H, n, block):
    row_ptr = torch.arange(H * n + 1, dtype=torch.int32) * n
    col = torch.arange(n, dtype=torch.int32).repeat(H * n)
    return losa.import_pattern(row_ptr, col, 1, H, n, block)


def gives_up_and_recovers(losa, call):
    """Calls with short limits, each followed by a normal one. Whether a wait
    runs out is the hardware's: a poll sleeps for a while before it fails, and
    a wait that ends in that time does not give up. Cold caches make the first
    waits long."""
    want = [t.clone() for t in call()]
    losa.check_status()
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    try:
        for limit in LIMITS:
            losa.set_wait_limit(limit)
            flush.fill_(limit & 1)
            call()
            try:
                losa.check_status()
            except losa.LosaError as e:
                assert e.status == -4
            losa.set_wait_limit(0)
            got = call()
            losa.check_status()
            for a, b in zip(want, got):
                assert torch.equal(a, b)
    finally:
        losa.set_wait_limit(0)


def tensors(H, n, block, d, dtype, count=4):
    g = torch.Generator("cuda").manual_seed(n + d)
    return [torch.randn(1, H, n * block, d, generator=g, device="cuda").to(dtype)
            for _ in range(count)]


@pytest.mark.parametrize("block,d", [(32, 64), (64, 64), (128, 64), (32, 128), (64, 128),
                                     (128, 128)])
@pytest.mark.parametrize("steps", [1, 2, 4])
def test_gradient_of_few_steps(losa, block, d, steps):
    H, n = 300, steps * 128 // block  # more tiles than SMs: others start on an SM at once
    pat = full_pattern(losa, H, n, block).prepare_backward()
    q, k, v, do = tensors(H, n, block, d, BF)
    o, lse = losa.sparse_attn(q, k, v, n * block, pat)
    gives_up_and_recovers(losa, lambda: losa.sparse_attn_bwd(q, k, v, o, lse, do, n * block, pat))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,d", [(32, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("steps", [1, 2])
def test_forward_of_few_steps(losa, block, d, steps, dtype):
    H, n = 301, steps * 128 // block
    pat = full_pattern(losa, H, n, block)
    q, k, v = tensors(H, n, block, d, dtype, 3)
    for call in (lambda: losa.sparse_attn(q, k, v, n * block, pat),
                 lambda: losa.dense_mass(q, k, v, n * block, block)):
        gives_up_and_recovers(losa, call)
