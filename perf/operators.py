"""Cases, plain forms and definitions of the training operators, for timing and comparison.

Two operators, each with its gradient direction:

  rope   rotary positions over the axes of a video token grid (time, height, width), read from the
         token-major tensors that a model's projections leave and written in the head-major, padded
         layout that the attention calls take ("pack"), and the way back for gradients ("unpack").
  bwd    the gradient of block-sparse attention over a frozen pattern, probabilities recomputed
         from the forward pass's row log-sum-exp.

`listed()` names fixed cases, `draw(rng)` gives more of the same ranges, `prepare` makes a case's
inputs on the GPU, `run` is one pass (elementary torch operations in 32 bits where `own` is False,
the package's calls where it is True), `exact` the same outputs from the definitions in 64 bits and
`work` the bytes and operations that a pass cannot do without.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases

def _rope(name, way, batch, heads, dim, grid, axes, block, dtype="bf16", text=0, start=(0, 0, 0),
          theta=10000.0, pairing="interleaved", fused=True, listed_positions=False):
    c = {"op": "rope", "way": way, "batch": batch, "heads": heads, "dim": dim, "block": block,
         "T": grid[0], "H": grid[1], "W": grid[2], "at": axes[0], "ah": axes[1], "aw": axes[2],
         "dtype": dtype, "text": text, "st": start[0], "sh": start[1], "sw": start[2],
         "theta": theta, "pairing": pairing, "fused": fused, "positions": listed_positions}
    return {"name": name, **c} if name else c


def _bwd(name, batch, heads, dim, tokens, block, kept, dtype="bf16"):
    c = {"op": "bwd", "batch": batch, "heads": heads, "dim": dim, "tokens": tokens,
         "block": block, "kept": kept, "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # The smallest workload of the repository: 256 tokens, two heads, fp32; a call's latency.
        _rope("rope_pack_tiny_fp32", "pack", 1, 2, 64, (4, 8, 8), (24, 20, 20), 32, "fp32"),
        # A Wan2.1-1.3B-shaped layer, views of one fused projection: an ordinary training step.
        _rope("rope_pack_wan2.1-1.3b", "pack", 1, 12, 128, (21, 30, 52), (44, 42, 42), 64),
        # The gradients of a CogVideoX-shaped layer (text tokens first, not rotated) on their way
        # back into one fused gradient.
        _rope("rope_unpack_cogvideox", "unpack", 1, 48, 64, (13, 30, 45), (16, 24, 24), 64,
              text=226),
        # The HunyuanVideo-shaped layer, the longest sequence.
        _rope("rope_pack_hunyuanvideo", "pack", 1, 24, 128, (33, 45, 80), (16, 56, 56), 128,
              theta=256.0),
        # A batch of two clips with listed positions (a later chunk of a long video), features
        # paired by halves, separate contiguous q, k, v, an odd grid.
        _rope("rope_pack_chunk_halves", "pack", 2, 16, 128, (5, 31, 27), (32, 48, 48), 64,
              start=(4096, 0, 0), pairing="halves", fused=False, listed_positions=True),
        # The smallest workload's gradient, fp32.
        _bwd("bwd_tiny_fp32", 1, 2, 64, 256, 32, 0.6, "fp32"),
        # A short clip: few tiles, a ragged last block.
        _bwd("bwd_short_clip", 1, 2, 128, 390, 64, 0.5),
        # A medium fp32 layer with a ragged end.
        _bwd("bwd_medium_fp32", 1, 4, 128, 2200, 64, 0.5, "fp32"),
        # A CogVideoX-shaped layer at the fraction of blocks that tau = 0.99 keeps.
        _bwd("bwd_cogvideox", 1, 48, 64, 17776, 64, 0.57),
        # A Wan2.1-1.3B-shaped layer.
        _bwd("bwd_wan2.1-1.3b", 1, 12, 128, 32760, 64, 0.62),
        # A batch of two at a low fraction kept (tau = 0.95), blocks of 32.
        _bwd("bwd_low_tau", 2, 8, 128, 16000, 32, 0.06),
        # One head of the HunyuanVideo-shaped layer (heads spread over GPUs), blocks of 128.
        _bwd("bwd_hunyuanvideo_head", 1, 1, 128, 118800, 128, 0.62),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dim = rng.choice([64, 128])
    block = rng.choice([32, 64, 128])
    if rng.random() < 0.5:
        # Up to the longest listed layer's values: batch * heads * tokens * dim.
        while True:
            grid = (_log(rng, 1, 40), _log(rng, 4, 60), _log(rng, 4, 90))
            batch, heads = rng.choice([1, 1, 2, 3]), _log(rng, 1, 48)
            text = rng.choice([0, 0, rng.randrange(1, 300)])
            if batch * heads * dim * (text + grid[0] * grid[1] * grid[2]) <= 24 * 128 * 118800:
                break
        half = dim // 2
        a = rng.randrange(2, half // 2)
        b = rng.randrange(2, half - a - 1)
        axes = (2 * a, 2 * b, 2 * rng.randrange(1, half - a - b + 1))
        return _rope(None, rng.choice(["pack", "unpack"]), batch, heads, dim, grid, axes, block,
                     rng.choice(["bf16", "bf16", "fp32"]), text,
                     (rng.randrange(0, 5000), rng.randrange(0, 64), rng.randrange(0, 64)),
                     rng.choice([256.0, 10000.0, 1000000.0]),
                     rng.choice(["interleaved", "halves"]), rng.random() < 0.6,
                     rng.random() < 0.3)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    # Scores of all pairs, before the pattern: at most those of the largest listed cases.
    most = 12 * 32760 ** 2 if dtype == "bf16" else 2 ** 28
    while True:
        tokens = _log(rng, 64, 60000 if dtype == "bf16" else 12000)
        batch, heads = rng.choice([1, 1, 2]), _log(rng, 1, 40)
        if batch * heads * tokens ** 2 <= most and (tokens + block - 1) // block <= 2047:
            break
    return _bwd(None, batch, heads, dim, tokens, block, round(rng.uniform(0.04, 1.0), 3), dtype)


# ------------------------------------------------------------------ inputs

def _tokens(c):
    return c["text"] + c["T"] * c["H"] * c["W"]


def _padded(c):
    n = _tokens(c) if c["op"] == "rope" else c["tokens"]
    return -(-n // c["block"]) * c["block"]


def _kept_counts(c):
    """How many key blocks each query block keeps: around kept * n, varying from row to row."""
    n = _padded(c) // c["block"]
    return [min(n, max(1, round(c["kept"] * n * (0.7 + 0.6 * ((I * 0.6180339887) % 1.0)))))
            for I in range(n)]


def _mask(c, g):
    """[B * H, n, n] kept blocks: the best-scoring key blocks of each query block, where scores are
    smooth over the sequence (near blocks, and bands of the same place in other frames) with some
    noise, as block masses are."""
    n, bh = _padded(c) // c["block"], c["batch"] * c["heads"]
    at = torch.arange(n, device="cuda", dtype=torch.float32)
    w = torch.rand(bh, 24, 1, generator=g, device="cuda") * 0.5
    phase = torch.rand(bh, 24, 1, generator=g, device="cuda") * 2 * math.pi
    f = torch.cos(w * at + phase)
    score = torch.einsum("bfi,bfj->bij", f, f) / 12
    score += 0.15 * torch.randn(bh, n, n, generator=g, device="cuda")
    count = torch.tensor(_kept_counts(c), device="cuda")
    order = score.argsort(-1, descending=True)
    mask = torch.zeros(bh, n, n, dtype=torch.bool, device="cuda")
    return mask.scatter_(2, order, (torch.arange(n, device="cuda") < count[:, None]).expand(bh, n, n))


def _rows(c, tokens):
    """Slices of query rows whose scores against all tokens fit into memory several times."""
    step = max(1, 2 ** 29 // tokens)
    return [slice(a, min(a + step, tokens)) for a in range(0, tokens, step)]


def _token_mask(state, h, rows):
    """The pattern of head h, by token."""
    b, L = state["case"]["block"], state["case"]["tokens"]
    i = torch.arange(rows.start, rows.stop, device="cuda") // b
    j = torch.arange(L, device="cuda") // b
    return state["mask"][h][i][:, j]


def _forward(state):
    """O (fp32, as the forward call gives it unless asked otherwise) and the row log-sum-exp."""
    c = state["case"]
    L, scale = c["tokens"], 1 / math.sqrt(c["dim"])
    q, k, v = (state[x].flatten(0, 1) for x in "qkv")
    o = torch.zeros_like(q, dtype=torch.float32)
    lse = torch.full(q.shape[:2], -math.inf, device="cuda")
    for h in range(q.shape[0]):
        kh, vh = k[h, :L].float(), v[h, :L].float()
        for r in _rows(c, L):
            s = (q[h, r].float() @ kh.T).mul_(scale)
            s.masked_fill_(~_token_mask(state, h, r), -math.inf)
            lse[h, r] = torch.logsumexp(s, 1)
            o[h, r] = s.sub_(lse[h, r, None]).exp_() @ vh
    shape = state["q"].shape
    return o.view(shape), lse.view(shape[:3])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = DTYPE[c["dtype"]]
    state = {"case": c}
    if c["op"] == "rope":
        L, B, H, d = _tokens(c), c["batch"], c["heads"], c["dim"]
        if c["way"] == "pack":
            # Projections' outputs: views of one fused tensor, or three of their own.
            if c["fused"]:
                x = torch.randn(B, L, 3, H, d, generator=g, device="cuda").to(t)
                state["x"] = tuple(x.unbind(2))
            else:
                state["x"] = tuple(torch.randn(B, L, H, d, generator=g, device="cuda").to(t)
                                   for _ in range(3))
        else:
            # The attention's gradients, zero in the padded rows.
            xs = []
            for _ in range(3):
                x = torch.zeros(B, H, _padded(c), d, device="cuda", dtype=t)
                x[:, :, :L] = torch.randn(B, H, L, d, generator=g, device="cuda") * 1e-2
                xs.append(x)
            state["x"] = tuple(xs)
        state["positions"] = None
        if c["positions"]:
            # Each clip of the batch at a place of its own in its video.
            p = _positions(c)[None].repeat(B, 1, 1)
            p[:, c["text"]:, 0] += torch.randint(0, 1000, (B, 1), generator=g, device="cuda",
                                                 dtype=torch.int32)
            state["positions"] = p
        if own:
            import block_sparse_attention_losa_b200 as losa
            state["losa"] = losa
            state["rope"] = losa.Rope((c["T"], c["H"], c["W"]), (c["at"], c["ah"], c["aw"]),
                                      theta=c["theta"], start=(c["st"], c["sh"], c["sw"]),
                                      n_text=c["text"], pairing=c["pairing"])
        return state
    # Attention: Q and K follow smooth features of the token's place plus noise, 2 % of the keys
    # take a shared direction (sinks); V is noise, the output's gradient small noise.
    B, H, L, Lp, d = c["batch"], c["heads"], c["tokens"], _padded(c), c["dim"]
    at = torch.arange(L, device="cuda", dtype=torch.float32)[:, None]
    w = torch.randn(B, H, 1, d, generator=g, device="cuda") * 0.01
    phase = torch.rand(B, H, 1, d, generator=g, device="cuda") * 2 * math.pi
    sink = torch.nn.functional.normalize(torch.randn(B, H, 1, d, generator=g, device="cuda"), dim=-1)
    is_sink = torch.rand(B, H, L, 1, generator=g, device="cuda") < 0.02
    for x in ("q", "k", "v", "do"):
        y = torch.randn(B, H, L, d, generator=g, device="cuda")
        if x in "qk":
            y = y * 0.5 + 1.5 * torch.cos(at * w + phase)
        if x == "k":
            y += is_sink * (3 * math.sqrt(d)) * sink
        if x == "do":
            y *= 1e-2
        state[x] = torch.zeros(B, H, Lp, d, device="cuda", dtype=t)
        state[x][:, :, :L] = y
    state["mask"] = _mask(c, g)
    state["o"], state["lse"] = _forward(state)
    if own:
        import block_sparse_attention_losa_b200 as losa
        m = state["mask"]
        row_ptr = torch.zeros(m.shape[0] * m.shape[1] + 1, dtype=torch.int32)
        row_ptr[1:] = m.sum(-1).flatten().cumsum(0)
        pat = losa.import_pattern(row_ptr, m.nonzero()[:, 2], B, H, m.shape[1], c["block"])
        pat.prepare_backward()
        state["losa"], state["pattern"] = losa, pat
    return state


# ------------------------------------------------------------------ one pass

def _positions(c):
    """[L, 3] int32 grid positions; text tokens stand at 0."""
    T, H, W = c["T"], c["H"], c["W"]
    i = torch.arange(T * H * W, device="cuda", dtype=torch.int32)
    p = torch.stack([i // (H * W) + c["st"], i // W % H + c["sh"], i % W + c["sw"]], 1)
    return torch.cat([torch.zeros(c["text"], 3, device="cuda", dtype=torch.int32), p])


def _turn(c, positions):
    """cos, sin [B or 1, L, 1, pairs] and the features (first, second) of each rotated pair."""
    p = (_positions(c)[None] if positions is None else positions).double()
    angle, first, second, at = [], [], [], 0
    for axis, n in enumerate((c["at"], c["ah"], c["aw"])):
        i = torch.arange(n // 2, device="cuda")
        angle.append(p[:, :, axis, None] * c["theta"] ** (-2.0 * i.double() / n))
        first.append(at + (2 * i if c["pairing"] == "interleaved" else i))
        second.append(at + (2 * i + 1 if c["pairing"] == "interleaved" else i + n // 2))
        at += n
    angle = torch.cat(angle, -1)
    angle[:, :c["text"]] = 0
    angle = angle[:, :, None]
    return angle.cos().float(), angle.sin().float(), torch.cat(first), torch.cat(second)


def _plain_rope(state):
    c = state["case"]
    L, Lp = _tokens(c), _padded(c)
    cos, sin, first, second = _turn(c, state["positions"])
    if c["way"] == "unpack":
        sin = -sin
    out = []
    for x, turned in zip(state["x"], (True, True, False)):
        if c["way"] == "unpack":
            x = x[:, :, :L].transpose(1, 2)
        y = x
        if turned:
            y = x.float()
            a, b = y[..., first], y[..., second]
            y = y.clone()
            y[..., first] = a * cos - b * sin
            y[..., second] = a * sin + b * cos
            y = y.to(x.dtype)
        if c["way"] == "pack":
            z = y.new_zeros(c["batch"], c["heads"], Lp, c["dim"])
            z[:, :, :L] = y.transpose(1, 2)
            y = z
        out.append(y)
    # Gradients of a fused projection come as one tensor [B, L, 3, H, d].
    if c["way"] == "unpack" and c["fused"]:
        return torch.stack(out, 2)
    return tuple(y.contiguous() for y in out)


def _plain_bwd(state):
    c = state["case"]
    L, scale = c["tokens"], 1 / math.sqrt(c["dim"])
    q, k, v, o, do = (state[x].flatten(0, 1) for x in ("q", "k", "v", "o", "do"))
    lse = state["lse"].flatten(0, 1)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    # Head by head and over slices of the query rows, since the scores of a whole layer (51 GB at
    # the Wan2.1-1.3B shape) do not fit beside their gradients.
    for h in range(q.shape[0]):
        kh, vh = k[h, :L].float(), v[h, :L].float()
        dkh, dvh = torch.zeros_like(kh), torch.zeros_like(vh)
        for r in _rows(c, L):
            qr, dor = q[h, r].float(), do[h, r].float()
            p = (qr @ kh.T).mul_(scale).sub_(lse[h, r, None]).exp_()
            p.masked_fill_(~_token_mask(state, h, r), 0)
            dvh += p.T @ dor
            ds = (dor @ vh.T).sub_((dor * o[h, r]).sum(1, keepdim=True)).mul_(p)
            dq[h, r] = (ds @ kh).mul_(scale).to(q.dtype)
            dkh += ds.T @ qr
        dk[h, :L], dv[h, :L] = dkh.mul_(scale).to(q.dtype), dvh.to(q.dtype)
    return tuple(x.view(state["q"].shape) for x in (dq, dk, dv))


def run(state):
    c = state["case"]
    if not own:
        return _plain_rope(state) if c["op"] == "rope" else _plain_bwd(state)
    losa = state["losa"]
    if c["op"] == "bwd":
        return losa.sparse_attn_bwd(state["q"], state["k"], state["v"], state["o"], state["lse"],
                                    state["do"], c["tokens"], state["pattern"])
    if c["way"] == "pack":
        return losa.rope_pack(*state["x"], c["block"], state["rope"],
                              positions=state["positions"])
    out = None
    if c["fused"]:
        fused = torch.empty(c["batch"], _tokens(c), 3, c["heads"], c["dim"], device="cuda",
                            dtype=state["x"][0].dtype)
        out = fused.unbind(2)
    got = losa.rope_unpack(*state["x"], _tokens(c), state["rope"], positions=state["positions"],
                           out=out)
    return fused if c["fused"] else got


# ------------------------------------------------------------------ definitions in 64 bits

def _exact_rope(state):
    """Each pair as a complex number times exp(i position theta^(-2 i / n)), or its conjugate."""
    c = state["case"]
    L = _tokens(c)
    pos = state["positions"]
    if pos is None:
        grid = torch.meshgrid(*(torch.arange(n, device="cuda") + s for n, s in
                                ((c["T"], c["st"]), (c["H"], c["sh"]), (c["W"], c["sw"]))),
                              indexing="ij")
        pos = torch.stack(grid, -1).reshape(1, -1, 3)
        pos = torch.nn.functional.pad(pos, (0, 0, c["text"], 0))
    is_text = (torch.arange(L, device="cuda") < c["text"])[None, :, None]
    out = []
    for n, x in enumerate(state["x"]):
        if c["way"] == "unpack":
            x = x[:, :, :L].permute(0, 2, 1, 3)
        parts, at = [], 0
        y = x.double()
        for axis, width in enumerate((c["at"], c["ah"], c["aw"])):
            seg = y[..., at:at + width]
            at += width
            if n == 2:
                parts.append(seg)
                continue
            freq = torch.exp(-math.log(c["theta"]) * torch.arange(0, width, 2, device="cuda",
                                                                  dtype=torch.float64) / width)
            turn = torch.where(is_text, 0.0, pos[..., axis, None].double() * freq)
            turn = torch.polar(torch.ones_like(turn), turn if c["way"] == "pack" else -turn)
            if c["pairing"] == "interleaved":
                z = torch.view_as_complex(seg.unflatten(-1, (width // 2, 2)).contiguous())
                parts.append(torch.view_as_real(z * turn[:, :, None]).flatten(-2))
            else:
                z = torch.complex(*(s.contiguous() for s in seg.chunk(2, -1))) * turn[:, :, None]
                parts.append(torch.cat([z.real, z.imag], -1))
        y = torch.cat(parts + [y[..., at:]], -1)
        if c["way"] == "pack":
            y = torch.nn.functional.pad(y.permute(0, 2, 1, 3), (0, 0, 0, _padded(c) - L))
        out.append(y.contiguous())
    return torch.stack(out, 2) if c["way"] == "unpack" and c["fused"] else tuple(out)


def _exact_bwd(state):
    """The softmax's Jacobian, from Q, K, V, the pattern and the output's gradient alone."""
    c = state["case"]
    L, b = c["tokens"], c["block"]
    shape = state["q"].shape
    grads = torch.zeros(3, *shape, device="cuda", dtype=torch.float64)
    flat = grads.view(3, -1, *shape[2:])
    blocks = torch.arange(L, device="cuda") // b
    for h in range(flat.shape[1]):
        q, k, v, do = (state[x].view(-1, *shape[2:])[h, :L].double() for x in ("q", "k", "v", "do"))
        q = q / math.sqrt(c["dim"])
        for a in range(0, L, max(1, 2 ** 28 // L)):
            r = slice(a, min(L, a + max(1, 2 ** 28 // L)))
            keep = state["mask"][h].index_select(0, blocks[r]).index_select(1, blocks)
            w = torch.where(keep, q[r] @ k.T, -math.inf)
            w = torch.softmax(w, -1)
            dw = do[r] @ v.T
            ds = dw.sub_(torch.linalg.vecdot(w, dw)[:, None]).mul_(w)
            flat[0, h, r] = ds @ k / math.sqrt(c["dim"])
            flat[1, h, :L] += ds.T @ q[r]
            flat[2, h, :L] += w.T @ do[r]
    return tuple(grads)


def exact(case, seed):
    c = case
    # About 20 seconds of 64-bit products and passes over the scores.
    if c["op"] == "bwd" and c["batch"] * c["heads"] * c["tokens"] ** 2 > 2 ** 34:
        return None
    state = prepare(c, seed)
    return _exact_rope(state) if c["op"] == "rope" else _exact_bwd(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    size = BYTES[c["dtype"]]
    if c["op"] == "rope":
        values = 3 * c["batch"] * c["heads"] * c["dim"]
        L, Lp = _tokens(c), _padded(c)
        turned = 2 * c["batch"] * c["heads"] * (c["at"] + c["ah"] + c["aw"]) * (L - c["text"])
        moved = values * size * (L + (Lp if c["way"] == "pack" else L))
        return {"bytes": moved + (12 * c["batch"] * L if c["positions"] else 0),
                "flops": 3 * turned}
    bh, L = c["batch"] * c["heads"], c["tokens"]
    pairs = bh * sum(_kept_counts(c)) * min(c["block"], L) ** 2
    # Q, K, V, dO, O (fp32) and lse in, dQ, dK, dV out; scores, dP, dV, dQ and dK are one product
    # each.
    return {"bytes": bh * L * (c["dim"] * (4 * size + 4) + 4) + bh * _padded(c) * c["dim"] * size * 3,
            "flops": 10 * pairs * c["dim"]}
