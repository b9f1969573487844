"""The training calls in autograd: backward() through them gives, bit for bit,
what the calls made by hand give (which test_gpu_backward.py and
test_gpu_rope.py hold to the formulas)."""
import pytest
import torch

from test_gpu_backward import BF, F32, make_mask, pattern_of

pytestmark = pytest.mark.gpu
B, H, d, grid, dims, block, L = 2, 3, 64, (2, 5, 13), (24, 20, 20), 64, 130


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


def setup(losa, dtype, seed=1):
    mask = make_mask(B * H, 3, 0.6, torch.Generator().manual_seed(2))
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(B, L, 3, H, d, generator=g, device="cuda").to(dtype)
    dout = torch.randn(B, L, H, d, generator=g, device="cuda").to(dtype)
    return pattern_of(losa, mask, B, H, block), losa.Rope(grid, dims), x, dout


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("listed", [False, True])
def test_layer(losa, dtype, listed):
    pat, rope, x, dout = setup(losa, dtype)
    pos = torch.randint(0, 99, (B, L, 3), device="cuda", dtype=torch.int32) if listed else None
    with torch.no_grad():
        want, state = losa.layer_attn(*x.unbind(2), rope, pat, positions=pos)
        grads = losa.layer_attn_bwd(dout, state)
    assert not want.requires_grad
    leaf = x.clone().requires_grad_()
    out, state = losa.layer_attn(*leaf.unbind(2), rope, pat, positions=pos)
    assert out.requires_grad and torch.equal(out, want)
    out.backward(dout)
    assert torch.equal(leaf.grad, torch.stack(grads, 2))
    # The state serves the call by hand all the same.
    for a, b in zip(losa.layer_attn_bwd(dout, state), grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_call_by_call(losa, dtype):
    pat, rope, x, dout = setup(losa, dtype)
    with torch.no_grad():
        out, state = losa.layer_attn(*x.unbind(2), rope, pat)
        grads = losa.layer_attn_bwd(dout, state)
    leaf = x.clone().requires_grad_()
    q, k, v = losa.rope_pack(*leaf.unbind(2), block, rope)
    o, lse = losa.sparse_attn(q, k, v, L, pat)
    assert not lse.requires_grad
    y = losa.rope_unpack(None, None, o, L, rope, out_dtype=dtype)[2]
    assert torch.equal(y, out)
    y.backward(dout)
    assert torch.equal(leaf.grad, torch.stack(grads, 2))


def test_parts_strides_and_repeats(losa):
    """Some inputs without gradients, a gradient of stride 0 (sum()), two
    backward passes over one graph, gradients that meet in one leaf."""
    pat, rope, x, dout = setup(losa, BF)
    q, k, v = (t.contiguous() for t in x.unbind(2))
    k.requires_grad_()
    out, state = losa.layer_attn(q, k, v, rope, pat)
    out.sum().backward(retain_graph=True)
    with torch.no_grad():
        want = losa.layer_attn_bwd(torch.ones_like(out), state)
    assert q.grad is None and v.grad is None and torch.equal(k.grad, want[1])
    k.grad = None
    out.backward(dout)
    with torch.no_grad():
        assert torch.equal(k.grad, losa.layer_attn_bwd(dout, state)[1])
    # One tensor as all three: the three gradients add up.
    one = q.clone().requires_grad_()
    out, state = losa.layer_attn(one, one, one, rope, pat)
    out.float().pow(2).sum().backward()
    with torch.no_grad():
        a, b, c = losa.layer_attn_bwd((2 * out.float()).to(BF), state)
        worst = (one.grad.float() - (a.float() + b.float() + c.float())).abs().max()
        # Two bf16 additions, half a step each.
        assert worst <= 2 * 2.0 ** -8 * (a.abs() + b.abs() + c.abs()).float().max()
    # A packed tensor that nothing uses, and one given alone.
    leaf = q.clone().requires_grad_()
    p, none, u = losa.rope_pack(leaf, None, leaf, block, rope)
    assert none is None
    p.float().sum().backward()
    with torch.no_grad():
        ones = torch.ones_like(p)
        assert torch.equal(leaf.grad, losa.rope_unpack(ones, None, None, L, rope)[0])


def test_padding_beyond_the_block(losa):
    """Unpacking from more padded rows than the block would give: the gradient
    has the input's rows, those past L zero."""
    rope = losa.Rope((33,), (64,))
    y = torch.randn(1, 2, 96, 64, device="cuda", requires_grad=True)
    out = losa.rope_unpack(y, None, None, 33, rope)[0]
    g = torch.randn(1, 33, 64, 2, device="cuda").transpose(2, 3)  # features not adjacent
    out.backward(g)
    want = losa.rope_pack(g.contiguous(), None, None, 32, rope)[0]
    assert torch.equal(y.grad[:, :, :64], want) and (y.grad[:, :, 64:] == 0).all()


def test_given_results_and_no_grad_stay_outside(losa):
    pat, rope, x, dout = setup(losa, BF)
    q, k, v = losa.rope_pack(*x.unbind(2), block, rope)
    assert not q.requires_grad
    q.requires_grad_()
    o = torch.empty(q.shape, device="cuda")
    got, lse = losa.sparse_attn(q, k, v, L, pat, o=o)
    assert got is o and not o.requires_grad
    with torch.no_grad():
        assert not losa.sparse_attn(q, k, v, L, pat)[0].requires_grad
    o2, none = losa.sparse_attn(q, k, v, L, pat, want_lse=False)
    assert none is None and torch.equal(o2, o) and o2.requires_grad


def test_other_stream_and_capture(losa):
    pat, rope, x, dout = setup(losa, BF)
    with torch.no_grad():
        out, state = losa.layer_attn(*x.unbind(2), rope, pat)
        want = torch.stack(losa.layer_attn_bwd(dout, state), 2)
    side = torch.cuda.Stream()
    leaf = x.clone().requires_grad_()
    side.wait_stream(torch.cuda.current_stream())
    y, _ = losa.layer_attn(*leaf.unbind(2), rope, pat, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    (got,) = torch.autograd.grad(y, leaf, dout)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del y, leaf, got
    static, sd = torch.zeros_like(x), torch.zeros_like(dout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        leaf = static.detach().requires_grad_()
        y, _ = losa.layer_attn(*leaf.unbind(2), rope, pat)
        (got,) = torch.autograd.grad(y, leaf, sd)
    static.copy_(x)
    sd.copy_(dout)
    graph.replay()
    assert torch.equal(got, want)


def test_pattern_not_prepared(losa):
    """Forward calls need no lists by key; the backward pass says so."""
    pat, rope, x, dout = setup(losa, BF)
    ex = pat.export("cpu")
    fresh = losa.import_pattern(ex["row_ptr"], ex["col_idx"], B, H, 3, block)
    leaf = x.clone().requires_grad_()
    out, _ = losa.layer_attn(*leaf.unbind(2), rope, fresh)
    with pytest.raises(losa.LosaError):
        out.backward(dout)
    fresh.prepare_backward()
    out, _ = losa.layer_attn(*leaf.unbind(2), rope, fresh)
    out.backward(dout)
    assert torch.isfinite(leaf.grad).all()
