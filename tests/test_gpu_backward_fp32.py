"""The fp32 gradient that forms lse and D itself, against the gradient's
formula in 64 bits, for keys with a large common part: in dQ that part stands
times sum_j dS_ij, which is 0 only if lse and D belong to the scores that P is
made of.

Tolerances are error bounds, value by value, u = 2^-24 (half a step of fp32).
The roundings of a sum of n terms are independent: their sum's deviation is
below sqrt(n / 3) u times the terms' sizes, and R(n) = (4 sqrt(n) + 8) u is
seven of those. |.| products bound the sizes.
  scores   es = R(d) scale |q||k|^T + 4 u |x| + 4 u |lse|, x the exponent
  l, D t   each term within ew = expm1(es) + 4 u of itself; a running sum is
           rescaled at most once a step, by an exponential (4 u) and a product,
           and joined over lanes likewise: in all within 8 R(n) of the sum
  lse      el = max_j ew + 8 R(n) + 4 u |lse|
  P        eP = P (expm1(es + el) + 4 u)
  dP       ep = R(d) |dO||V|^T
  D        eD = sum_j P (ew |dP| + ep) + (max_j ew + 16 R(n)) sum_j P |dP|
  dS       e = P (ep + eD) + eP |dP - D|
  dQ       scale (e |K| + R(n) |dS||K|), dK likewise, dV eP |dO| + R(n) P |dO|,
plus half a step of the result's type.
"""
import math

import pytest
import torch

from test_gpu_backward import close, make_mask, pattern_of, token_mask

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


def reference(q, k, v, do, keep, scale):
    """Gradients in 64 bits ([BH, L, d] each) and their error bounds."""
    d, L = q.shape[2], q.shape[1]
    t = lambda x: x.transpose(1, 2)
    s = torch.where(keep, (q @ t(k)) * scale, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    x = torch.where(keep, s - lse, 0.0)
    p = torch.where(keep, torch.exp(x), 0.0)
    dp = do @ t(v)
    dd = dp - (p * dp).sum(-1, keepdim=True)
    ds = p * dd
    R = lambda terms: (4 * math.sqrt(terms) + 8) * U
    n = R(L)
    es = R(d) * scale * (q.abs() @ t(k.abs())) + 4 * U * (x.abs() + lse.abs())
    es = torch.where(keep, es, 0.0)
    ew = torch.expm1(es) + 4 * U
    worst = ew.max(-1, keepdim=True)[0]
    el = worst + 8 * n + 4 * U * lse.abs()
    eP = p * (torch.expm1(es + el) + 4 * U)
    ep = R(d) * (do.abs() @ t(v.abs()))
    eD = (p * (ew * dp.abs() + ep)).sum(-1, keepdim=True) + \
        (worst + 16 * n) * (p * dp.abs()).sum(-1, keepdim=True)
    e = p * (ep + eD) + eP * dd.abs()
    pairs = [(ds @ k * scale, (e @ k.abs() + n * (ds.abs() @ k.abs())) * scale),
             (t(ds) @ q * scale, (t(e) @ q.abs() + n * (t(ds.abs()) @ q.abs())) * scale),
             (t(p) @ do, t(eP) @ do.abs() + n * (t(p) @ do.abs()))]
    return [a for a, _ in pairs], [b for _, b in pairs]


def inputs(B, H, L, d, common, do_dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    q, k, v, do = torch.randn(4, B * H, L, d, generator=g, device="cuda")
    k = k + common * torch.randn(B * H, 1, d, generator=g, device="cuda")
    return q, k, v, do.to(do_dtype)


def padded(x, B, H, Lp):
    y = torch.full((B, H, Lp, x.shape[2]), float("nan"), device="cuda", dtype=x.dtype)
    y[:, :, :x.shape[1]] = x.view(B, H, *x.shape[1:])
    return y


SHAPES = [  # B, H, d, L, block, density
    (1, 1, 64, 1, 32, 1.0), (1, 2, 128, 33, 32, 0.6), (2, 1, 64, 129, 128, 1.0),
    (1, 2, 128, 390, 64, 0.5), (1, 1, 64, 1000, 32, 0.2),
    (1, 4, 128, 700, 64, 0.5), (2, 3, 64, 500, 128, 0.6),  # 24 tiles: the 128-thread kernels
    (1, 3, 64, 1100, 32, 0.3),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("do_dtype,out_dtype", [(F32, F32), (BF, F32), (F32, BF)])
def test_gradients_without_o_and_lse(losa, shape, do_dtype, out_dtype):
    B, H, d, L, block, density = shape
    n = -(-L // block)
    mask = make_mask(B * H, n, density, torch.Generator().manual_seed(L))
    pat = pattern_of(losa, mask, B, H, block)
    x = inputs(B, H, L, d, 3.0, do_dtype, L + d)
    q, k, v, do = (padded(t, B, H, n * block) for t in x)
    ref, tol = reference(*(t.double() for t in x), token_mask(mask, block, L).cuda(),
                         1 / math.sqrt(d))
    got = losa.sparse_attn_bwd(q, k, v, None, None, do, L, pat, out_dtype=out_dtype)
    close(got, ref, tol, L)
    again = losa.sparse_attn_bwd(q, k, v, None, None, do, L, pat, out_dtype=out_dtype)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("common", [0.0, 3.0, 10.0])
def test_layer(losa, common):
    """layer_attn and layer_attn_bwd in fp32, tokens that are not turned (so
    that packing is exact): the forward call runs in tf32, the gradients are
    those of fp32 all the same."""
    B, H, L, d, block = 1, 2, 400, 128, 64
    mask = make_mask(B * H, 7, 0.6, torch.Generator().manual_seed(3))
    pat = pattern_of(losa, mask, B, H, block)
    x = inputs(B, H, L, d, common, F32, 12)
    ref, tol = reference(*(t.double() for t in x), token_mask(mask, block, L).cuda(),
                         1 / math.sqrt(d))
    q, k, v, do = (t.view(B, H, L, d).transpose(1, 2) for t in x)
    rope = losa.Rope((0,), (d,), n_text=L)
    _, state = losa.layer_attn(q, k, v, rope, pat)
    got = [t.transpose(1, 2) for t in losa.layer_attn_bwd(do, state)]
    losa.check_status()
    close(got, ref, tol, L)


def test_extreme_rows(losa):
    """Scores of either sign up to some 600, so that running sums are rescaled
    to nothing, and rows that keep one block of which one key is valid."""
    H, d, L, block = 2, 64, 257, 64
    mask = torch.ones(H, 5, 5, dtype=torch.bool)
    mask[:, 2] = False
    mask[:, 2, 4] = True
    pat = pattern_of(losa, mask, 1, H, block)
    q, k, v, do = inputs(1, H, L, d, 0.0, F32, 5)
    q = q * torch.linspace(1e-3, 60.0, L, device="cuda")[None, :, None]
    ref, tol = reference(*(t.double() for t in (q, k, v, do)), token_mask(mask, block, L).cuda(),
                         1 / math.sqrt(d))
    got = losa.sparse_attn_bwd(*(padded(t, 1, H, 320) for t in (q, k, v)), None, None,
                               padded(do, 1, H, 320), L, pat)
    close(got, ref, tol, L)


def test_graph_and_stream(losa):
    H, d, L, block = 2, 64, 200, 32
    mask = make_mask(H, 7, 0.5, torch.Generator().manual_seed(3))
    pat = pattern_of(losa, mask, 1, H, block)
    a, b = ([padded(t, 1, H, 224) for t in inputs(1, H, L, d, 3.0, BF, s)] for s in (1, 2))
    call = lambda x, **kw: losa.sparse_attn_bwd(*x[:3], None, None, x[3], L, pat, **kw)
    want = [call(a), call(b)]
    static = [t.clone() for t in a]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(static)
    for x, w in zip((a, b), want):
        for s, t in zip(static, x):
            s.copy_(t)
        graph.replay()
        assert all(torch.equal(i, j) for i, j in zip(got, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moved = call(a, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(moved, want[0]))


def test_refusals(losa):
    H, d, L, block = 2, 64, 200, 32
    mask = make_mask(H, 7, 0.5, torch.Generator().manual_seed(3))
    pat = pattern_of(losa, mask, 1, H, block)
    q, k, v, do = (padded(t, 1, H, 224) for t in inputs(1, H, L, d, 0.0, F32, 1))
    lse = torch.zeros(1, H, 224, device="cuda")
    for args in ((q, k, v, q, None, do), (q, k, v, None, lse, do),
                 (q.to(BF), k.to(BF), v.to(BF), None, None, do)):
        with pytest.raises(ValueError):
            losa.sparse_attn_bwd(*args, L, pat)
    lib = losa.lib()
    out = [torch.empty_like(q) for _ in range(3)]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()
    for dtype, o, l in ((1, q, None), (1, None, lse), (0, None, None)):
        assert lib.losa_sparse_attn_bwd(p(q), p(k), p(v), dtype, p(o), 1, p(l), p(do), 1, d, L, 0.1,
                                        pat.handle, *map(p, out), 1, p(ws), 1 << 20, None) == -1
