"""losa_rope_pack and losa_rope_unpack against plain rotations in 64 bits.

Tolerance, per value, with u = 2^-24 and (x, y) the turned pair: the turn is
rounded once to fp32 (at most half a turn: pi * u of angle), sine and cosine
are within 2 u of their values there, and one product and one fused
multiply-add round: (|x| + |y|) (pi + 2 + 2) u, below 8 u (|x| + |y|). A bf16
result adds half a step, 2^-8 of the value. Values that are not turned are
copied (one rounding where the output has fewer bits).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def losa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import block_sparse_attention_losa_b200 as m
    return m


def positions_of(grid, start, n_text):
    """[L, axes] int64 positions of a grid's tokens, text tokens at 0."""
    axes = torch.meshgrid(*(torch.arange(n) + s for n, s in zip(grid, start)), indexing="ij")
    p = torch.stack([a.reshape(-1) for a in axes], 1)
    return torch.cat([torch.zeros(n_text, len(grid), dtype=torch.int64), p])


def turn64(x, pos, dims, theta, scale, n_text, pairing, sign):
    """x [B, L, H, d] (fp64, CPU) turned; also the per-value |x| + |y|."""
    y, size = x.clone(), x.abs()
    at = 0
    pos = pos.double()
    for a, n in enumerate(dims):
        for i in range(n // 2):
            f, g = (at + 2 * i, at + 2 * i + 1) if pairing == "interleaved" else \
                (at + i, at + i + n // 2)
            ang = sign * pos[..., a] * scale[a] * theta ** (-2.0 * i / n)
            ang = torch.where(torch.arange(x.shape[1]) < n_text, torch.zeros_like(ang), ang)
            c, s = ang.cos()[..., None], ang.sin()[..., None]
            y[..., f] = x[..., f] * c - x[..., g] * s
            y[..., g] = x[..., f] * s + x[..., g] * c
            size[..., f] = size[..., g] = x[..., f].abs() + x[..., g].abs()
        at += n
    return y, size


def close(got, ref, size):
    got = got.detach().cpu()
    tol = 8 * U * size
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    worst = ((got.double() - ref).abs() - tol).max().item()
    assert worst <= 0, worst


CASES = [  # B, H, d, grid, dims, n_text, start, scale, theta, block
    (1, 2, 64, (4, 8, 8), (24, 20, 20), 0, (0, 0, 0), (1.0, 1.0, 1.0), 1e4, 32),
    (2, 3, 128, (3, 5, 7), (44, 42, 42), 3, (5, 0, 2), (1.0, 0.5, 2.0), 1e4, 64),
    (1, 1, 128, (1, 1, 1), (16, 56, 56), 0, (0, 0, 0), (1.0, 1.0, 1.0), 256.0, 128),
    (1, 5, 64, (9, 13), (16, 32), 0, (0, 7), (1.0, 1.0), 1e4, 32),
    (3, 2, 128, (131,), (64,), 1, (2 ** 31 - 140,), (1.0,), 1e6, 64),
    (1, 2, 64, (2, 3, 11), (32, 16, 16), 66, (100000, -50, 3), (1.0, 1.0, 1.0), 1e4, 64),
    (1, 40, 128, (1, 2, 9), (32, 48, 48), 0, (0, 0, 0), (1.0, 1.0, 1.0), 1e4, 32),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("din,dout", [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16"),
                                      ("bf16", "fp32")])
def test_pack_and_unpack(losa, case, pairing, din, dout):
    B, H, d, grid, dims, n_text, start, scale, theta, block = case
    L = math.prod(grid) + n_text
    Lp = -(-L // block) * block
    g = torch.Generator().manual_seed(L * 7 + d)
    rope = losa.Rope(grid, dims, theta=theta, start=start, scale=scale, n_text=n_text,
                     pairing=pairing)
    pos = positions_of(grid, start, n_text)[None]
    # Views of one fused tensor, as a fused projection gives.
    x = torch.randn(B, L, 3, H, d, generator=g).to(DT[din])
    xg = x.cuda()
    got = losa.rope_pack(*xg.unbind(2), block, rope, out_dtype=DT[dout])
    for t in range(3):
        src = x[:, :, t].double()
        ref, size = turn64(src, pos, dims, theta, scale, n_text, pairing, 1) if t < 2 else \
            (src, 0 * src)
        assert got[t].shape == (B, H, Lp, d) and got[t].dtype == DT[dout]
        close(got[t][:, :, :L].transpose(1, 2), ref, size)
        assert (got[t][:, :, L:] == 0).all()
    # And back, into the views of one fused gradient; padded rows hold NaN.
    y = torch.randn(3, B, H, Lp, d, generator=g).to(DT[din])
    y[:, :, :, L:] = float("nan")
    fused = torch.full((B, L, 3, H, d), 7.0, device="cuda", dtype=DT[dout])
    losa.rope_unpack(*y.cuda().unbind(0), L, rope, out=fused.unbind(2))
    for t in range(3):
        src = y[t][:, :, :L].transpose(1, 2).double()
        ref, size = turn64(src, pos, dims, theta, scale, n_text, pairing, -1) if t < 2 else \
            (src, 0 * src)
        close(fused[:, :, t], ref, size)


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("layout", ["token", "head", "odd", "broadcast"])
def test_strides_and_listed_positions(losa, pairing, layout):
    """Head-major and unaligned views, a broadcast batch, and positions far
    apart listed per token, which stand for grid and start."""
    B, H, L, d, dims = 2, 3, 45, 64, (20, 22, 22)
    g = torch.Generator().manual_seed(3)
    if layout == "token":
        x = torch.randn(B, L, H, d, generator=g).bfloat16().cuda()
    elif layout == "head":
        x = torch.randn(B, H, L, d, generator=g).bfloat16().cuda().transpose(1, 2)
    elif layout == "odd":  # rows of 65 elements from element 1 on: 2-byte alignment
        x = torch.randn(B, L, H, 65, generator=g).bfloat16().cuda()[..., 1:]
    else:
        x = torch.randn(1, L, H, d, generator=g).bfloat16().cuda().expand(B, L, H, d)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, L, 3), generator=g, dtype=torch.int64)
    rope = losa.Rope((1, 1, 1), dims, theta=100.0, start=(9, 9, 9), n_text=4, pairing=pairing)
    q, none, v = losa.rope_pack(x, None, x, 32, rope, positions=pos.int().cuda())
    assert none is None
    ref, size = turn64(x.cpu().double(), pos, dims, 100.0, (1.0,) * 3, 4, pairing, 1)
    # A position of 2^31 in fp64 turns is exact to 2^31 2^-53 * 2 pi < 2e-6 of
    # angle in the reference and in the kernel each.
    got = q[:, :, :L].transpose(1, 2).cpu().double()
    tol = (8 * U + 4e-6) * size + 2.0 ** -8 * (ref.abs() + 4e-6 * size)
    assert ((got - ref).abs() <= tol).all()
    assert torch.equal(v[:, :, :L].transpose(1, 2), x)
    out = torch.empty_strided((B, L, H, d), (L * H * 67 + 5, H * 67, 67, 1), dtype=torch.float32,
                              device="cuda") if layout == "odd" else None
    back = losa.rope_unpack(None, q, None, L, rope, positions=pos.int().cuda(),
                            out_dtype=torch.float32, out=None if out is None else (None, out, None))
    ref, size = turn64(q[:, :, :L].transpose(1, 2).cpu().double(), pos, dims, 100.0, (1.0,) * 3, 4,
                       pairing, -1)
    assert ((back[1].cpu().double() - ref).abs() <= (8 * U + 4e-6) * size).all()


def test_text_alone_and_single_tokens(losa):
    """A sequence of text tokens only is moved, not turned; one token of a
    later chunk turns by its own position."""
    x = torch.randn(2, 5, 3, 64, device="cuda").bfloat16()
    rope = losa.Rope((0, 3, 3), (16, 24, 24), n_text=5)
    q, k, v = losa.rope_pack(x, x, x, 32, rope)
    for y in (q, k, v):
        assert torch.equal(y[:, :, :5].transpose(1, 2), x) and (y[:, :, 5:] == 0).all()
    one = torch.randn(1, 1, 2, 128, device="cuda")
    for pairing in ("interleaved", "halves"):
        rope = losa.Rope((1, 1, 1), (44, 42, 42), start=(1234567, 9, 77), pairing=pairing)
        y = losa.rope_pack(one, None, None, 32, rope)[0][:, :, :1].transpose(1, 2)
        ref, size = turn64(one.cpu().double(), torch.tensor([[[1234567, 9, 77]]]), (44, 42, 42),
                           1e4, (1.0,) * 3, 0, pairing, 1)
        close(y, ref, size)


def test_untouched_neighbours_and_infinities(losa):
    """A fused gradient's other columns stay as they are; features that no
    axis turns pass infinities and NaN through unchanged."""
    B, H, L, d = 1, 2, 33, 64
    rope = losa.Rope((33,), (32,))
    y = torch.randn(B, H, 64, d, device="cuda")
    y[0, 0, 3, 40] = float("inf")
    y[0, 1, 4, 33] = float("nan")
    buf = torch.full((B, L, 4, H, d), 5.0, device="cuda")
    losa.rope_unpack(y, None, None, L, rope, out=(buf[:, :, 1], None, None))
    assert (buf[:, :, [0, 2, 3]] == 5).all()
    same = buf[:, :, 1, :, 32:].transpose(1, 2)
    assert torch.equal(same.nan_to_num(123.0), y[:, :, :L, 32:].nan_to_num(123.0))
    assert torch.isfinite(buf[0, :, 1, :, :32]).all()


def test_unpack_is_the_gradient_of_pack(losa):
    """<pack(x), y> = <x, unpack(y)> for fp32 (the rotation's transpose), to
    the sums' rounding in 64 bits of products that are within 16 u."""
    B, H, L, d = 2, 4, 70, 128
    rope = losa.Rope((2, 5, 7), (44, 42, 42), pairing="halves")
    x = [torch.randn(B, L, H, d, device="cuda") for _ in range(3)]
    y = [torch.randn(B, H, 96, d, device="cuda") for _ in range(3)]
    px = losa.rope_pack(*x, 32, rope)
    uy = losa.rope_unpack(*y, L, rope)
    for a, b, c, e in zip(px, y, x, uy):
        lhs = (a.double() * b.double()).sum()
        rhs = (c.double() * e.double()).sum()
        bound = 32 * U * (a.double().abs() * b.double().abs()).sum()
        assert (lhs - rhs).abs() <= 2 * bound


def test_streams_graphs_and_repeats(losa):
    B, H, L, d = 1, 6, 390, 128
    rope = losa.Rope((3, 10, 13), (44, 42, 42))
    x = torch.randn(B, L, 3, H, d, device="cuda").bfloat16()
    want = losa.rope_pack(*x.unbind(2), 64, rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = losa.rope_pack(*x.unbind(2), 64, rope, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    static = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        out = losa.rope_pack(*static.unbind(2), 64, rope)
        back = losa.rope_unpack(*out, L, rope)
    static.copy_(x)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    eager = losa.rope_unpack(*want, L, rope)
    assert all(torch.equal(a, b) for a, b in zip(eager, back))


def test_binding_refusals(losa):
    rope = losa.Rope((2, 3, 4), (16, 24, 24))
    x = torch.zeros(1, 24, 2, 64, device="cuda")
    y = torch.zeros(1, 2, 32, 64, device="cuda")
    bad = [
        lambda: losa.rope_pack(x, x[:, :23], x, 32, rope),
        lambda: losa.rope_pack(x, x.bfloat16(), x, 32, rope),
        lambda: losa.rope_pack(x, x, x, 48, rope),
        lambda: losa.rope_pack(x.transpose(2, 3), None, None, 32, rope),
        lambda: losa.rope_pack(x, x, None, 32, rope, out=(y, None, None)),
        lambda: losa.rope_pack(x, None, None, 32, rope, out=(y[:, :, :31], None, None)),
        lambda: losa.rope_pack(x, x, x, 32, rope, positions=torch.zeros(1, 24, 3, device="cuda")),
        lambda: losa.rope_pack(x, x, x, 32, rope,
                               positions=torch.zeros(1, 23, 3, device="cuda", dtype=torch.int32)),
        lambda: losa.rope_unpack(y.transpose(0, 1).expand(2, 2, 32, 64), None, None, 24, rope),
        lambda: losa.rope_unpack(y, None, None, 24, rope, out=(x.bfloat16(), None, None),
                                 out_dtype=torch.float32),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: losa.rope_pack(x[:, :23], None, None, 32, rope),  # grid has 24 tokens
                 lambda: losa.rope_unpack(y, None, None, 33, rope),
                 lambda: losa.rope_unpack(y, None, None, 24, rope,
                                          out=(x[:, :1].expand(1, 24, 2, 64), None, None))):
        with pytest.raises(losa.LosaError):
            call()
    with pytest.raises(TypeError):
        losa.rope_pack(x.half(), None, None, 32, rope)


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_text_after_the_video_by_listed_positions(losa, pairing):
    """Listed positions of zero turn nothing; the video's tokens in front turn
    as on their grid."""
    B, H, d, grid, dims, text = 2, 2, 64, (2, 3, 4), (16, 24, 24), 7
    n = math.prod(grid)
    pos = torch.zeros(B, n + text, 3, dtype=torch.int32)
    pos[:, :n] = positions_of(grid, (0, 0, 0), 0)
    x = torch.randn(B, n + text, H, d, device="cuda").bfloat16()
    q = losa.rope_pack(x, None, None, 32, losa.Rope((0, 0, 0), dims, pairing=pairing),
                       positions=pos.cuda())[0].transpose(1, 2)
    assert torch.equal(q[:, n:n + text], x[:, n:])
    alone = losa.rope_pack(x[:, :n], None, None, 32, losa.Rope(grid, dims, pairing=pairing))[0]
    assert torch.equal(q[:, :n], alone.transpose(1, 2)[:, :n])
