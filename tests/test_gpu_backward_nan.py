"""A NaN in one row of an input reaches the gradients that depend on it: that
row's dQ and, over the keys that the row keeps, dK and (not for O) dV. Rows of
other heads stay finite."""
import pytest
import torch

from test_gpu_backward import BF, F32, make_mask, pattern_of, token_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", ["o", "lse", "do"])
@pytest.mark.parametrize("L,row", [(300, 0), (300, 9), (300, 170), (300, 299), (1, 0), (4200, 33)])
def test_nan_reaches_the_gradients(losa, dtype, which, L, row):
    H, d, block = 2, 64, 64
    n = -(-L // block)
    mask = make_mask(H, n, 0.5, torch.Generator().manual_seed(L))
    pat = pattern_of(losa, mask, 1, H, block)
    g = torch.Generator("cuda").manual_seed(L + row)
    q, k, v, do = torch.randn(4, 1, H, n * block, d, generator=g, device="cuda").to(dtype)
    o, lse = losa.sparse_attn(q, k, v, L, pat)
    dict(o=o, do=do, lse=lse[..., None])[which][0, 1, row, -1] = float("nan")
    dq, dk, dv = (t[0] for t in losa.sparse_attn_bwd(q, k, v, o, lse, do, L, pat))
    losa.check_status()
    kept = token_mask(mask, block, L)[1, row].cuda()
    bad = lambda t: ~torch.isfinite(t)
    assert bad(dq[1, row]).all()
    assert bad(dk[1, :L][kept]).all()
    if which == "lse":
        assert bad(dv[1, :L][kept]).all()
    if which == "do":
        assert bad(dv[1, :L, -1][kept]).all()
    for t in (dq, dk, dv):
        assert torch.isfinite(t[0]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", ["q", "k", "v", "o", "lse", "do"])
def test_padded_rows_of_the_gradients_stay_zero(losa, dtype, which):
    L, H, d, block = 300, 2, 64, 64
    pat = pattern_of(losa, torch.ones(H, 5, 5, dtype=torch.bool), 1, H, block)
    q, k, v, do = torch.randn(4, 1, H, 320, d, device="cuda").to(dtype)
    o, lse = losa.sparse_attn(q, k, v, L, pat)
    dict(q=q, k=k, v=v, o=o, lse=lse[..., None], do=do)[which][0, 1, 290, -1] = float("nan")
    for t in losa.sparse_attn_bwd(q, k, v, o, lse, do, L, pat):
        assert (t[:, :, L:] == 0).all()
    losa.check_status()
