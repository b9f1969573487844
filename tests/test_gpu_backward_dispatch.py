"""The gradient's kernels on both sides of each rule that chooses among them,
every head dim, block size and result type, against the 64-bit formula with
test_gpu_backward.py's bounds:
  bf16  heads of 32 and of 33 tiles of 128 rows (dQ with and without dS's
        remainder), and short heads in a call of more than 32 tiles;
  fp32  calls of 20 and of 21 tiles (256 and 128 threads a CTA)."""
import pytest
import torch

from test_gpu_backward import BF, F32, close, inputs, make_mask, pattern_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


def check(losa, B, H, L, d, block, density, dtype, do_dtype, out_dtype):
    n = -(-L // block)
    mask = make_mask(B * H, n, density, torch.Generator().manual_seed(L + block))
    pat = pattern_of(losa, mask, B, H, block)
    args, ref, tol = inputs(B, H, L, n * block, d, dtype, F32, do_dtype, mask, block, L + d)
    got = losa.sparse_attn_bwd(*args, L, pat, out_dtype=out_dtype)
    losa.check_status()
    close(got, ref, tol, L)
    pat.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("H,L,head_tiles", [(1, 4090, 32), (1, 4117, 33), (34, 150, 2)])
def test_bf16(losa, d, block, out_dtype, H, L, head_tiles):
    assert -(-L // 128) == head_tiles and (L > 4000 or H * head_tiles > 32)
    check(losa, 1, H, L, d, block, 0.3, BF, BF, out_dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("B,H,L,tiles", [(2, 2, 630, 20), (1, 3, 850, 21)])
def test_fp32(losa, d, block, out_dtype, B, H, L, tiles):
    assert B * H * -(-L // 128) == tiles
    check(losa, B, H, L, d, block, 0.5, F32, F32, out_dtype)
