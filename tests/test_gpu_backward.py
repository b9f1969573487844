"""losa_sparse_attn_bwd against the gradient's formula in 64 bits, and the
forward pass's own differences.

The reference takes the call's own inputs (O and lse among them) in 64 bits.
Tolerances are error bounds, value by value, with u = 2^-24 (half a step of
fp32), v = 2^-8 (half a step of bf16) on the tensor-core path and 0 on the
fp32 one, and |.| products for sums (a sum of n terms in fp32 is within n u of
the sum of their sizes):
  scores   es = (d + 4) u scale |q||k|^T + 4 u |x| + 4 u |lse|, x the exponent
  P        eP = P (expm1(es) + 4 u); rounded to bf16 as an operand: + v P
  dP - D   ed = (d + 4) u (|dO||V|^T + |dO|.|O|)
  dS       eS = eP' |dP - D| + P ed; rounded: + v |dS|
  dV       sum(eP |dO|) + (n + 8) u sum(P |dO|),  dQ, dK likewise of dS,
plus half a step of the result's type. eP' is eP without the operand's
rounding: dS is formed from the unrounded P.
"""
import math

import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
V = 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


def make_mask(bh, n, density, g, unused=False):
    """Kept blocks, ragged from row to row, at least one each; with `unused`
    the second key block is kept by no query block."""
    mask = torch.rand(bh, n, n, generator=g) < density * (0.3 + 1.4 * torch.rand(bh, n, 1,
                                                                               generator=g))
    mask[:, torch.arange(n), torch.randint(0, n, (n,), generator=g)] = True
    if unused and n > 1:
        mask[:, :, 1] = False
        mask[:, :, 0] |= ~mask.any(-1)
    return mask


def pattern_of(losa, mask, B, H, block):
    row_ptr = torch.zeros(mask.shape[0] * mask.shape[1] + 1, dtype=torch.int32)
    row_ptr[1:] = mask.sum(-1).flatten().cumsum(0)
    return losa.import_pattern(row_ptr, mask.nonzero()[:, 2], B, H, mask.shape[1],
                               block).prepare_backward()


def token_mask(mask, block, L):
    return mask.repeat_interleave(block, 1).repeat_interleave(block, 2)[:, :L, :L]


def forward64(q, k, v, keep, scale):
    s = (q @ k.transpose(1, 2)) * scale
    s = torch.where(keep, s, -math.inf)
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[..., None]) @ v, lse


def reference(q, k, v, o, lse, do, keep, scale, rounded):
    """Gradients in 64 bits ([BH, L, d] each) and their error bounds."""
    d, L = q.shape[2], q.shape[1]
    r = V if rounded else 0.0
    t = lambda x: x.transpose(1, 2)
    x = (q @ t(k)) * scale - lse[..., None]
    p = torch.where(keep, torch.exp(x), 0.0)
    es = (d + 4) * U * scale * (q.abs() @ t(k.abs())) + 4 * U * (x.abs() + lse.abs()[..., None])
    ep = p * (torch.expm1(es) + 4 * U)
    dd = (do @ t(v)) - (do * o).sum(-1, keepdim=True)
    ed = (d + 4) * U * (do.abs() @ t(v.abs()) + (do * o).abs().sum(-1, keepdim=True))
    ds = p * dd
    es_ = ep * dd.abs() + p * ed
    es_ = es_ + r * (ds.abs() + es_)
    ep = ep + r * (p + ep)
    n = (L + 8) * U
    return [(ds @ k * scale, (es_ @ k.abs() + n * (ds.abs() @ k.abs())) * scale),
            (t(ds) @ q * scale, (t(es_) @ q.abs() + n * (t(ds.abs()) @ q.abs())) * scale),
            (t(p) @ do, t(ep) @ do.abs() + n * (t(p) @ do.abs()))]


def close(got, ref, tol, L, names=("dq", "dk", "dv")):
    for name, g, (r, e) in zip(names, got, zip(ref, tol)):
        step = V if g.dtype == BF else U
        e = e * (1 + step) + step * r.abs()
        x = g.flatten(0, 1)
        worst = ((x[:, :L].double() - r).abs() - e).max().item()
        assert worst <= 0, (name, worst, r.abs().max().item())
        assert (x[:, L:] == 0).all(), name


def inputs(B, H, L, Lp, d, dtype, o_dtype, do_dtype, mask, block, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(4, B * H, L, d, generator=g).to("cuda")
    x[0] *= spread
    q, k, v = (t.to(dtype).double() for t in x[:3])
    do = x[3].to(do_dtype).double()
    keep = token_mask(mask, block, L).cuda()
    scale = 1 / math.sqrt(d)
    o, lse = forward64(q, k, v, keep, scale)
    o, lse = o.to(o_dtype).double(), lse.float().double()

    def padded(t, dt, fill=float("nan")):  # rows >= L must not matter
        y = torch.full((B * H, Lp) + t.shape[2:], fill, device="cuda", dtype=dt)
        y[:, :L] = t.to(dt)
        return y.view(B, H, Lp, *t.shape[2:])

    args = [padded(q, dtype), padded(k, dtype), padded(v, dtype), padded(o, o_dtype),
            padded(lse, F32, -math.inf), padded(do, do_dtype)]
    # The tensor cores read a fp32 dO rounded to bf16.
    seen = do.to(BF).double() if dtype == BF else do
    pairs = reference(q, k, v, o, lse, seen, keep, scale, dtype == BF)
    return args, [p[0] for p in pairs], [p[1] for p in pairs]


SHAPES = [  # B, H, d, L, block, density
    (1, 1, 64, 1, 32, 1.0), (1, 2, 128, 1, 128, 1.0), (2, 1, 128, 31, 32, 1.0),
    (1, 2, 64, 33, 32, 0.5), (1, 1, 128, 64, 64, 1.0), (1, 2, 128, 129, 128, 0.6),
    (1, 2, 64, 256, 32, 0.5), (2, 3, 128, 390, 64, 0.4), (1, 2, 64, 500, 128, 0.5),
    (1, 1, 128, 721, 32, 0.15), (1, 2, 64, 1000, 64, 0.3), (3, 1, 128, 1025, 128, 0.7),
    (1, 1, 64, 1100, 32, 0.05),
]
TYPES = [(BF, F32, BF, BF), (BF, BF, BF, F32), (BF, F32, F32, BF), (F32, F32, F32, F32),
         (F32, BF, BF, F32), (F32, F32, F32, BF)]  # in, o, do, out


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("types", TYPES)
def test_gradients(losa, shape, types):
    B, H, d, L, block, density = shape
    dtype, o_dtype, do_dtype, out_dtype = types
    n = -(-L // block)
    mask = make_mask(B * H, n, density, torch.Generator().manual_seed(L), unused=L % 2 == 0)
    pat = pattern_of(losa, mask, B, H, block)
    args, ref, tol = inputs(B, H, L, n * block, d, dtype, o_dtype, do_dtype, mask, block, L + d)
    got = losa.sparse_attn_bwd(*args, L, pat, out_dtype=out_dtype)
    losa.check_status()
    assert all(t.dtype == out_dtype for t in got)
    close(got, ref, tol, L)
    if n > 1 and L % 2 == 0:  # a key block that nothing keeps
        for t in got[1:]:
            assert (t[:, :, block:2 * block] == 0).all()
    again = losa.sparse_attn_bwd(*args, L, pat, out_dtype=out_dtype)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    pat.close()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_flat_and_peaked_rows(losa, dtype, spread):
    """Scores that are all alike, and rows where one key takes everything."""
    B, H, d, L, block = 1, 2, 128, 300, 64
    mask = make_mask(2, 5, 0.6, torch.Generator().manual_seed(1))
    pat = pattern_of(losa, mask, B, H, block)
    args, ref, tol = inputs(B, H, L, 320, d, dtype, F32, dtype, mask, block, 5, spread)
    close(losa.sparse_attn_bwd(*args, L, pat), ref, tol, L)
    losa.check_status()


@pytest.mark.parametrize("block,d,L", [(32, 64, 33), (64, 128, 64), (128, 64, 97), (32, 128, 90)])
def test_dq_of_small_calls(losa, block, d, L):
    """In calls of few rows dQ takes dS with 16 bits, so that what the keys
    have in common cancels: here all share a long part and some a longer
    one."""
    B, H, n = 1, 2, -(-L // block)
    g = torch.Generator().manual_seed(d + L)
    mask = make_mask(B * H, n, 0.8, g)
    pat = pattern_of(losa, mask, B, H, block)
    x = torch.randn(4, B * H, L, d, generator=g).to("cuda")
    x[0] *= 0.1
    x[1] += 3 * torch.randn(B * H, 1, d, generator=g).to("cuda")
    x[1, :, ::9] += 10 * torch.randn(B * H, 1, d, generator=g).to("cuda")
    q, k, v, do = x.to(BF).double()
    keep, scale, t = token_mask(mask, block, L).cuda(), 1 / math.sqrt(d), lambda y: y.transpose(1, 2)
    o, lse = forward64(q, k, v, keep, scale)
    o, lse = o.float().double(), lse.float().double()
    z = (q @ t(k)) * scale - lse[..., None]
    p = torch.where(keep, torch.exp(z), 0.0)
    dd = (do @ t(v)) - (do * o).sum(-1, keepdim=True)
    ds = p * dd
    # A term of a tensor-core sum is off by at most a step (2 U) of the sum of
    # magnitudes, one of D's fp32 sum by U; the exponential by 3.1e-7 < 6 U and
    # its argument's roundings; dS by V of what its rounding left, V of it; dQ
    # sums 2 L terms.
    es = 2 * (d + 4) * U * scale * (q.abs() @ t(k.abs())) + 4 * U * (z.abs() + lse.abs()[..., None])
    ed = (d + 4) * U * (2 * do.abs() @ t(v.abs()) + (do * o).abs().sum(-1, keepdim=True))
    e = p * (torch.expm1(es) + 8 * U) * dd.abs() + p * ed
    e = e + V * V * (ds.abs() + e)
    tol = scale * (e @ k.abs() + 4 * (L + 8) * U * (ds.abs() @ k.abs()))

    def padded(y, dt):
        z = torch.zeros((B * H, n * block) + y.shape[2:], device="cuda", dtype=dt)
        z[:, :L] = y.to(dt)
        return z.view(B, H, n * block, *y.shape[2:])

    dq = losa.sparse_attn_bwd(padded(q, BF), padded(k, BF), padded(v, BF), padded(o, F32),
                              padded(lse, F32), padded(do, BF), L, pat, out_dtype=F32)[0]
    want = scale * (ds @ k)
    got = dq.flatten(0, 1)[:, :L].double()
    assert ((got - want).abs() - tol * (1 + U) - U * want.abs()).max().item() <= 0
    # dS rounded once would be off by more than that.
    once = scale * (ds.to(BF).double() @ k)
    assert ((once - want).abs() - tol).max().item() > 0
    losa.check_status()


@pytest.mark.parametrize("block,d", [(32, 64), (64, 128), (128, 128), (32, 128), (128, 64)])
def test_lists_by_key_are_the_transposed_pattern(losa, block, d):
    B, H, n = 2, 2, 21
    mask = make_mask(4, n, 0.3, torch.Generator().manual_seed(block), unused=True)
    pat = pattern_of(losa, mask, B, H, block)
    ex = pat.export_backward()
    per, tiles = 128 // block, -(-n * block // 128)
    counts = []
    for t in range(4 * tiles):
        bh, kt = divmod(t, tiles)
        m = mask[bh][:, kt * per:(kt + 1) * per]
        want = [(I, sum(int(x) << c for c, x in enumerate(m[I].tolist())))
                for I in range(n) if m[I].any()]
        got = ex["key_entry"][ex["key_ptr"][t]:ex["key_ptr"][t + 1]].tolist()
        assert [(e & 0xFFFF, e >> 16) for e in got] == want
        counts.append(len(want))
    order = ex["key_order"].tolist()
    assert sorted(order) == list(range(4 * tiles))
    for a, b in zip(order, order[1:]):
        assert a // tiles < b // tiles or (a // tiles == b // tiles and counts[a] >= counts[b])


def test_long_ragged_pattern(losa):
    """Many iterations per tile, several key tiles, a ragged end; bf16."""
    B, H, d, L, block = 1, 1, 128, 5003, 64
    n = -(-L // block)
    mask = make_mask(1, n, 0.5, torch.Generator().manual_seed(9))
    pat = pattern_of(losa, mask, B, H, block)
    args, ref, tol = inputs(B, H, L, n * block, d, BF, F32, BF, mask, block, 11)
    close(losa.sparse_attn_bwd(*args, L, pat), ref, tol, L)
    losa.check_status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_against_differences_of_the_forward_call(losa, dtype):
    """The loss <O, R> of the forward call moves as the gradients say: a
    central difference along random directions. bf16 / tf32 forward outputs
    carry rounding noise, so the step is large and the bound is the noise over
    the step: O's errors are below 1e-2 each (the forward's own tolerance)
    but of random sign; their sum against R (norm |R|) over a step h stays
    below 6 * 1e-3 |R| / h, 1e-3 being the forward's bound on their mean size;
    the quadratic and cubic terms are below 5 % of the derivative's scale."""
    wl = W.custom("bwd", 2, 64, (2, 8, 16), 32, text_tokens=3, amplitude=1.0, seed=77)
    L = wl.seq_len
    q, k, v = (t.cuda() for t in W.generate(wl, dtype=F32))
    q, k, v = (t.to(dtype) for t in (q, k, v))
    _, _, mass = losa.dense_mass(q, k, v, L, 32)
    pat = losa.select(mass, 32, 0.95).prepare_backward()
    g = torch.Generator("cuda").manual_seed(2)
    R = torch.randn(q.shape, generator=g, device="cuda").to(dtype)
    R[:, :, L:] = 0
    o, lse = losa.sparse_attn(q, k, v, L, pat)
    grads = losa.sparse_attn_bwd(q, k, v, o, lse, R, L, pat, out_dtype=F32)
    h = 0.25
    for i in range(3):
        w = torch.randn(q.shape, generator=g, device="cuda")
        w[:, :, L:] = 0
        w *= 4.0 / w.norm()
        ends = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = (x[i].float() + sign * h * w).to(dtype)
            step = x[i].double() - (q, k, v)[i].double()
            ends.append(((losa.sparse_attn(*x, L, pat)[0].double() * R.double()).sum(), step))
        moved = ends[0][1] - ends[1][1]
        want = (grads[i].double() * moved).sum()
        got = ends[0][0] - ends[1][0]
        size = (grads[i].double().norm() * moved.norm()).item()
        assert (got - want).abs().item() <= 12e-3 * R.double().norm().item() + 0.05 * size


def plain_layer(x, mask, block, grid, dims):
    """The layer in 64 bits, differentiable: x [B, L, 3, H, d] projections."""
    B, L, _, H, d = x.shape
    pos = torch.stack(torch.meshgrid(*(torch.arange(m, device="cuda") for m in grid),
                                     indexing="ij"), -1).reshape(-1, 3).double()
    ang = torch.cat([pos[:, a, None] * 10000.0 ** (-torch.arange(0, m, 2, device="cuda") / m)
                     for a, m in enumerate(dims)], 1)[None, :, None]
    qkv = torch.view_as_complex(x.unflatten(-1, (d // 2, 2)))
    turn = torch.polar(torch.ones_like(ang), ang)
    q, k = (torch.view_as_real(qkv[:, :, i] * turn).flatten(-2).transpose(1, 2) for i in (0, 1))
    v = x[:, :, 2].transpose(1, 2)
    keep = token_mask(mask, block, L).cuda().view(B, H, L, L)
    s = torch.where(keep, q @ k.transpose(2, 3) / math.sqrt(d), -math.inf)
    return (torch.softmax(s, -1) @ v).transpose(1, 2)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_training_step(losa, whole, dtype):
    """pack, forward, backward and unpack as a training step runs them, call
    by call and through layer_attn and layer_attn_bwd: the gradients with
    respect to the token-major projections against a plain formulation's, and
    (bf16, whose forward call allocates nothing of its own) two captured
    steps' bits against the eager one's."""
    B, H, d, grid, dims, block, L = 2, 3, 128, (3, 10, 13), (44, 42, 42), 64, 390
    rope = losa.Rope(grid, dims)
    g = torch.Generator("cuda").manual_seed(4)
    n = -(-L // block)
    mask = make_mask(B * H, n, 0.5, torch.Generator().manual_seed(6))
    pat = pattern_of(losa, mask, B, H, block)
    x = torch.randn(B, L, 3, H, d, generator=g, device="cuda").to(dtype)
    dout = torch.randn(B, L, H, d, generator=g, device="cuda").to(dtype)

    def step(x, dout):
        dx = torch.empty_like(x)
        if whole:
            out, state = losa.layer_attn(*x.unbind(2), rope, pat)
            losa.layer_attn_bwd(dout, state, out=dx.unbind(2))
            return out, dx
        q, k, v = losa.rope_pack(*x.unbind(2), block, rope)
        o, lse = losa.sparse_attn(q, k, v, L, pat)
        out = losa.rope_unpack(None, None, o, L, rope, out_dtype=dtype)[2]
        do = losa.rope_pack(None, None, dout, block, rope)[2]
        grads = losa.sparse_attn_bwd(q, k, v, o, lse, do, L, pat)
        losa.rope_unpack(*grads, L, rope, out=dx.unbind(2))
        return out, dx

    out, dx = step(x, dout)
    losa.check_status()
    y = x.double().requires_grad_()
    ref = plain_layer(y, mask, block, grid, dims)
    ref.backward(dout.double())
    # bf16: roundings on the way of a gradient: q and k, P, dS, dq/dk, dx, each
    # at most 2^-8 of its value; they add as norms, and q and k's also through
    # the scores (|s| up to 5 here, e^(5 * 2^-8)): below 8 half steps. fp32:
    # the forward call's operands and weights are tf32 (half a step 2^-11),
    # which reaches the gradient through O and lse: the same count of those.
    unit = V if dtype == BF else 2.0 ** -11
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    assert rel(out, ref) <= 8 * unit
    assert rel(dx, y.grad) <= 8 * unit
    if dtype != BF:
        return
    static, sd = torch.zeros_like(x), torch.zeros_like(dout)
    graphs = []
    for _ in range(2):  # two captured steps, each with its own memory
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(static, sd)
        graphs.append((graph, got))
    static.copy_(x)
    sd.copy_(dout)
    for graph, _ in graphs:
        graph.replay()
    for _, (o2, dx2) in graphs:
        assert torch.equal(o2, out) and torch.equal(dx2, dx)


def test_layer_on_another_stream_and_positions(losa):
    """The whole layer on a side stream, with positions listed per clip that
    repeat the grid's, gives the default stream's bits."""
    B, H, d, grid, block, L = 2, 2, 64, (2, 5, 9), 32, 90
    mask = make_mask(B * H, 3, 0.7, torch.Generator().manual_seed(2))
    pat = pattern_of(losa, mask, B, H, block)
    rope = losa.Rope(grid, (16, 24, 24))
    x = torch.randn(B, L, 3, H, d, device="cuda").to(BF)
    dout = torch.randn(B, L, H, d, device="cuda").to(BF)
    out, state = losa.layer_attn(*x.unbind(2), rope, pat)
    want = losa.layer_attn_bwd(dout, state)
    pos = torch.stack(torch.meshgrid(*(torch.arange(m) for m in grid), indexing="ij"),
                      -1).reshape(1, -1, 3).int().repeat(B, 1, 1).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, state2 = losa.layer_attn(*x.unbind(2), rope, pat, positions=pos, stream=side)
    got = losa.layer_attn_bwd(dout, state2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, out2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_layer_with_positions_alone(losa):
    """Listed positions stand for the grid: the rope's own may be another."""
    B, H, d, block, L = 2, 2, 64, 32, 90
    mask = make_mask(B * H, 3, 0.7, torch.Generator().manual_seed(2))
    pat = pattern_of(losa, mask, B, H, block)
    x = torch.randn(B, L, 3, H, d, device="cuda").to(BF)
    dout = torch.randn(B, L, H, d, device="cuda").to(BF)
    pos = torch.randint(0, 50, (B, L, 3), device="cuda", dtype=torch.int32)
    both = []
    for grid in ((2, 5, 9), (4, 4, 4)):
        out, state = losa.layer_attn(*x.unbind(2), losa.Rope(grid, (16, 24, 24)), pat,
                                     positions=pos)
        both.append((out, *losa.layer_attn_bwd(dout, state)))
    assert all(torch.equal(a, b) for a, b in zip(*both))


def test_offsets_past_32_bits(losa):
    """A layer of more than 2^31 elements a tensor: its first and last heads
    give the bits that they give alone."""
    B, H, d, block, n = 3, 22, 128, 128, 2047
    L = n * block - 26
    assert B * H * L * d > 2 ** 31
    mask = torch.zeros(B * H, n, n, dtype=torch.bool)
    i = torch.arange(n)
    mask[:, i, i] = mask[:, i, n - 1 - i] = True
    pat, one = pattern_of(losa, mask, B, H, block), pattern_of(losa, mask[:1], 1, 1, block)
    rope = losa.Rope((L,), (d,))
    x = torch.empty(B, L, 3, H, d, device="cuda", dtype=BF).normal_()
    dout = torch.empty(B, L, H, d, device="cuda", dtype=BF).normal_()
    dx = torch.empty_like(x)
    out, state = losa.layer_attn(*x.unbind(2), rope, pat)
    losa.layer_attn_bwd(dout, state, out=dx.unbind(2))
    del state
    for b, h in ((0, 0), (B - 1, H - 1)):
        y, state = losa.layer_attn(*(t[b:b + 1, :, h:h + 1] for t in x.unbind(2)), rope, one)
        assert torch.equal(out[b:b + 1, :, h:h + 1], y)
        got = losa.layer_attn_bwd(dout[b:b + 1, :, h:h + 1], state)
        for t, g in enumerate(got):
            assert torch.equal(dx[b:b + 1, :, t, h:h + 1], g)
    losa.check_status()


def test_a_wait_that_runs_out(losa):
    """With a wait limit of one cycle the call gives up, the status says so,
    and the next call is whole again."""
    B, H, d, L, block = 1, 2, 128, 1000, 64
    mask = make_mask(2, 16, 0.5, torch.Generator().manual_seed(8))
    pat = pattern_of(losa, mask, B, H, block)
    args, ref, tol = inputs(B, H, L, 1024, d, BF, F32, BF, mask, block, 31)
    try:
        losa.set_wait_limit(1)
        losa.sparse_attn_bwd(*args, L, pat)
        with pytest.raises(losa.LosaError) as e:
            losa.check_status()
        assert e.value.status == -4
    finally:
        losa.set_wait_limit(0)
    close(losa.sparse_attn_bwd(*args, L, pat), ref, tol, L)
    losa.check_status()


def test_two_streams_at_once(losa):
    B, H, d, L, block = 1, 4, 128, 1000, 64
    mask = make_mask(4, 16, 0.5, torch.Generator().manual_seed(8))
    pat = pattern_of(losa, mask, B, H, block)
    a, _, _ = inputs(B, H, L, 1024, d, BF, F32, BF, mask, block, 21)
    b, _, _ = inputs(B, H, L, 1024, d, BF, F32, BF, mask, block, 22)
    want = [losa.sparse_attn_bwd(*x, L, pat) for x in (a, b)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [losa.sparse_attn_bwd(*x, L, pat, stream=s) for x, s in zip((a, b), side)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("flip", [False, True])
def test_uneven_warps(losa, d, flip):
    """Blocks of 32 in a checkerboard in which every second pair of a step's
    four blocks is kept by one block of a tile only: some warps of a tile skip
    all their arithmetic, others none, over many steps, so that they drift as
    far apart as the kernel lets them."""
    B, H, L, block = 1, 3, 1984, 32
    n = L // block
    i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
    mask = torch.where(j % 4 < 2, i % 4 == 3, i % 4 != 3)
    if flip:
        mask = mask.T | (i == j)
    mask = mask | (j == i // 4 * 4)
    mask = mask[None].repeat(H, 1, 1)
    pat = pattern_of(losa, mask, B, H, block)
    args, ref, tol = inputs(B, H, L, L, d, BF, F32, BF, mask, block, 41)
    for _ in range(3):
        got = losa.sparse_attn_bwd(*args, L, pat)
        losa.check_status()
        close(got, ref, tol, L)


def test_lists_by_key_on_another_stream_than_the_selection(losa):
    """The lists by key built on a side stream right after a selection on the
    default one, whose list writes may still be running."""
    g = torch.Generator("cuda").manual_seed(1)
    mass = torch.rand(1, 8, 512, 512, generator=g, device="cuda")
    mass /= mass.sum(-1, keepdim=True)
    want = losa.select(mass, 64, 0.9).prepare_backward().export_backward()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        pat = losa.select(mass, 64, 0.9).prepare_backward(stream=side)
        got = pat.export_backward()
        assert torch.equal(want["key_ptr"], got["key_ptr"])
        assert torch.equal(want["key_entry"], got["key_entry"])
        pat.close()


def test_given_outputs_and_workspace(losa):
    B, H, d, L, block = 1, 2, 64, 200, 32
    mask = make_mask(2, 7, 0.5, torch.Generator().manual_seed(3))
    pat = pattern_of(losa, mask, B, H, block)
    args, ref, tol = inputs(B, H, L, 224, d, BF, BF, BF, mask, block, 2)
    out = [torch.full(args[0].shape, 9.0, device="cuda") for _ in range(3)]
    need = losa.lib().losa_sparse_attn_bwd_workspace(pat.handle, 0, 0, d)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    got = losa.sparse_attn_bwd(*args, L, pat, dq=out[0], dk=out[1], dv=out[2], workspace=ws)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(out, got))
    assert (ws[need:] == 255).all()
    close(got, ref, tol, L)


def test_refusals(losa):
    B, H, d, L, block = 1, 2, 64, 200, 32
    mask = make_mask(2, 7, 0.5, torch.Generator().manual_seed(3))
    pat = pattern_of(losa, mask, B, H, block)
    q, k, v, o, lse, do = inputs(B, H, L, 224, d, BF, BF, BF, mask, block, 2)[0]
    for change in (dict(o=o[:, :, :200]), dict(lse=lse.double()), dict(lse=lse[:, :, :200]),
                   dict(do=do.transpose(0, 1)), dict(q=q[:, :1]), dict(do=do.cpu()),
                   dict(dq=o.float(), dk=o), dict(dv=o[..., ::2]), dict(q=q.float()),
                   dict(workspace=torch.empty(1 << 20))):
        a = dict(q=q, k=k, v=v, o=o, lse=lse, do=do, L=L, pattern=pat)
        a.update(change)
        with pytest.raises(ValueError):
            losa.sparse_attn_bwd(**a)
    with pytest.raises(TypeError):
        losa.sparse_attn_bwd(q, k, v, o.half(), lse, do, L, pat)
    for change in (dict(L=192), dict(L=225), dict(L=0), dict(scale=0.0),
                   dict(scale=float("nan")),
                   dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        a = dict(q=q, k=k, v=v, o=o, lse=lse, do=do, L=L, pattern=pat)
        a.update(change)
        with pytest.raises(losa.LosaError):
            losa.sparse_attn_bwd(**a)
    for change in (dict(dq=q), dict(dv=do), dict(dq=o, dk=o), dict(dk=q, dv=k)):
        a = dict(q=q, k=k, v=v, o=o, lse=lse, do=do, L=L, pattern=pat)
        a.update(change)
        with pytest.raises(losa.LosaError):
            losa.sparse_attn_bwd(**a)
    need = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    bits = [torch.empty_like(q) for _ in range(3)]
    ptr = [t.data_ptr() for t in (q, k, v, o, lse, do, *bits, need)]
    assert losa.lib().losa_sparse_attn_bwd(  # lse halfway into an element
        *ptr[:3], 0, ptr[3], 0, ptr[4] + 2, ptr[5], 0, d, L, 0.1, pat.handle, *ptr[6:9], 0, ptr[9],
        1 << 20, None) == -1
    fresh = losa.import_pattern(*(pat.export("cpu")[x] for x in ("row_ptr", "col_idx")), B, H, 7,
                                block, device="cuda")
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        with pytest.raises(losa.LosaError):
            fresh.prepare_backward(stream=stream)
        torch.zeros(1, device="cuda")  # the capture goes on
    with pytest.raises(losa.LosaError):  # not prepared
        losa.sparse_attn_bwd(q, k, v, o, lse, do, L, fresh)
    with pytest.raises(losa.LosaError):
        fresh.export_backward()
    fresh.prepare_backward().prepare_backward()  # twice is once
    losa.sparse_attn_bwd(q, k, v, o, lse, do, L, fresh)
    losa.check_status()
    fresh.close()
    with pytest.raises(ValueError):
        losa.sparse_attn_bwd(q, k, v, o, lse, do, L, fresh)
