"""A head's gradient does not depend on the heads beside it: the bits of a
batch of heads are those of each head alone, on both sides of every rule by
which the gradient's kernels are chosen."""
import pytest
import torch

from test_gpu_backward import make_mask, pattern_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


@pytest.mark.parametrize("B,H,L,d,block", [
    (1, 48, 90, 64, 32), (2, 20, 64, 128, 64), (1, 40, 128, 128, 128), (1, 33, 31, 128, 32),
    (1, 12, 500, 64, 128), (1, 20, 700, 128, 64), (1, 3, 4096, 64, 64), (1, 2, 4225, 128, 128),
])
def test_a_head_alone_and_in_a_batch(losa, B, H, L, d, block):
    n = -(-L // block)
    assert B * H * -(-L // 128) > 32
    mask = make_mask(B * H, n, 0.5, torch.Generator().manual_seed(L))
    g = torch.Generator("cuda").manual_seed(L + d)
    q, k, v, do = torch.randn(4, B, H, n * block, d, generator=g, device="cuda").to(BF)
    pat = pattern_of(losa, mask, B, H, block)
    o, lse = losa.sparse_attn(q, k, v, L, pat)
    whole = losa.sparse_attn_bwd(q, k, v, o, lse, do, L, pat)
    losa.check_status()
    for b, h in ((0, 0), (B - 1, H // 2), (B - 1, H - 1)):
        i = b * H + h
        one = pattern_of(losa, mask[i:i + 1], 1, 1, block)
        args = [x[b:b + 1, h:h + 1] for x in (q, k, v, o, lse, do)]
        for a, w in zip(losa.sparse_attn_bwd(*args, L, one), whole):
            assert torch.equal(a, w[b:b + 1, h:h + 1])
