"""What is measured of the operators around a hybrid layer's linear layers and
token mixers:

* ``quantize`` -- E4M3 codes with a float32 scale for each 1 x 128 piece of a
  row (activations) or each 128 x 128 block (weights).
* ``linear`` -- a linear layer on such a weight: dense activations are
  quantized by row pieces and multiplied block by block.
* ``rope`` -- query and key heads: RMS norm per head and the position rotation,
  with one or three position axes, in one pass.
* ``conv`` -- the short causal convolution along the tokens of each channel,
  for prompts and single tokens, with the state that it keeps per sequence.
* ``step`` -- the gated delta rule for the next tokens of many sequences, each
  with its state in a pool.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    """Each case says what it stands for."""
    def quantize(name, rows, cols, block, dtype):
        return dict(name=name, op="quantize", rows=rows, cols=cols, block=block, dtype=dtype)

    def linear(name, m, n, k, dtype):
        return dict(name=name, op="linear", m=m, n=n, k=k, dtype=dtype)

    def rope(name, tokens, q_heads, k_heads, dim, rotary, axes, far, dtype, norm=True, pairs="half", offset=False):
        return dict(name=name, op="rope", tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim, rotary=rotary, axes=axes,
                    far=far, dtype=dtype, norm=norm, pairs=pairs, offset=offset)

    def conv(name, seqs, longest, channels, width, dtype, silu=True, bias=False, fresh=False):
        return dict(name=name, op="conv", seqs=seqs, longest=longest, channels=channels, width=width, dtype=dtype, silu=silu,
                    bias=bias, fresh=fresh)

    def step(name, batch, q_len, k_heads, v_heads, dtype, empty=False, fresh=False):
        return dict(name=name, op="step", batch=batch, q_len=q_len, k_heads=k_heads, v_heads=v_heads, dtype=dtype, empty=empty,
                    fresh=fresh)

    return [
        # the activation of a long prompt's down projection
        quantize("quantize rows 8192x17408", 8192, 17408, 1, "bf16"),
        # a float32 weight of odd size, once when a checkpoint is loaded
        quantize("quantize blocks 1000x2064", 1000, 2064, 128, "f32"),
        # a decode step of three sequences through the widest projection: bound by the weight's bytes
        linear("linear 3x34816x5120", 3, 34816, 5120, "bf16"),
        # a small mixed batch (a chunk and some single tokens)
        linear("linear 200x5120x17408", 200, 5120, 17408, "bf16"),
        # float32 in and out, odd sizes: columns that end inside a scale's block, rows inside a tile
        linear("linear 77x1000x2064 f32", 77, 1000, 2064, "f32"),
        # a long prompt's down projection: bound by the matrix products
        linear("linear 8192x5120x17408", 8192, 5120, 17408, "bf16"),
        # a decode step of 64 sequences far into their contexts, a quarter of each wide head rotated
        rope("rope step 64, 24+4 x 256", 64, 24, 4, 256, 64, 3, 262144, "bf16", offset=True),
        # a prompt of text and images
        rope("rope prompt 16384, 32+8 x 128", 16384, 32, 8, 128, 128, 3, 32768, "bf16"),
        # a decode step: one token of each of 64 sequences, one of the places empty
        conv("conv step 64x1, 10240", 64, 1, 10240, 4, "bf16"),
        # prompts of unequal lengths in one batch, an empty one among them
        conv("conv 7 prompts to 9000, 10240", 7, 9000, 10240, 4, "bf16", bias=True, fresh=True),
        # one conversation's next token
        step("step 1x1, 16/48 heads", 1, 1, 16, 48, "bf16"),
        # the decode step of a full batch
        step("step 64x1, 16/48 heads", 64, 1, 16, 48, "bf16", empty=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        dtype = "f32" if rng.random() < 0.25 else "bf16"
        op = rng.choice(["quantize", "linear", "linear", "rope", "conv", "step"])
        if op == "quantize":
            c = dict(op=op, rows=_log(rng, 1, 16384), cols=16 * _log(rng, 1, 2176), block=rng.choice([1, 1, 128]), dtype=dtype)
            if c["rows"] * c["cols"] > 8192 * 17408:
                continue
        elif op == "linear":
            c = dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 64, 34816), k=16 * _log(rng, 8, 1088), dtype=dtype)
            if rng.random() < 0.5:  # most widths are whole blocks
                c["n"], c["k"] = -(-c["n"] // 128) * 128, -(-c["k"] // 128) * 128
            if c["m"] * c["n"] * c["k"] > (8192 * 5120 * 17408 if dtype == "bf16" else 8192 * 5120 * 17408 // 4):
                continue
        elif op == "rope":
            dim, k_heads = rng.choice([64, 128, 128, 256]), rng.randint(1, 8)
            c = dict(op=op, tokens=_log(rng, 1, 32768), q_heads=k_heads * rng.randint(1, 8), k_heads=k_heads, dim=dim,
                     rotary=rng.choice([dim, dim // 2, dim // 4]), axes=rng.choice([1, 3]), far=_log(rng, 64, 1 << 20), dtype=dtype,
                     norm=rng.random() < 0.8, pairs=rng.choice(["half", "half", "next"]), offset=rng.random() < 0.4)
            if c["tokens"] * (c["q_heads"] + k_heads) * dim * _DT[dtype].itemsize > 16384 * 40 * 128 * 2:
                continue
        elif op == "conv":
            c = dict(op=op, seqs=_log(rng, 1, 256), longest=_log(rng, 1, 32768), channels=8 * _log(rng, 8, 1280),
                     width=rng.choice([2, 3, 4, 4]), dtype=dtype, silu=rng.random() < 0.8, bias=rng.random() < 0.5,
                     fresh=rng.random() < 0.4)
            if sum(_lens(c)) * c["channels"] * _DT[dtype].itemsize > 33000 * 10240 * 2:
                continue
        else:
            k_heads = _log(rng, 1, 16)
            c = dict(op=op, batch=_log(rng, 1, 256), q_len=rng.choice([1, 1, 1, rng.randint(2, 8)]), k_heads=k_heads,
                     v_heads=k_heads * rng.randint(1, 4), dtype=dtype, empty=rng.random() < 0.4, fresh=rng.random() < 0.3)
            if c["batch"] * c["v_heads"] > 64 * 48 or c["batch"] * c["v_heads"] * c["q_len"] > 3 * 64 * 48:
                continue
        return c


def _lens(c):
    """Tokens of each sequence of a convolution: one each, or spread over [0, longest] in an order that is not sorted."""
    n, top = c["seqs"], c["longest"]
    if top == 1 or n == 1:
        return [top] * n
    turn = next(s for s in range(max(1, n * 5 // 8), 2 * n + 2) if math.gcd(s, n) == 1)
    return [top * (b * turn % n) // (n - 1) for b in range(n)]


def _empty(c):
    """The places of a padded batch that hold no sequence."""
    return {c["batch"] // 2} if c["empty"] and c["batch"] > 1 else set()


def work(case):
    c = case
    size = _DT[c["dtype"]].itemsize
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (size + 1) + 4 * -(-c["rows"] // c["block"]) * -(-c["cols"] // 128), "flops": 3 * n}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m * k + m * n) * size + n * k + 4 * -(-n // 128) * -(-k // 128), "flops": 2 * m * n * k}
    if c["op"] == "rope":
        n = c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["dim"]
        return {"bytes": 2 * n * size + 8 * c["axes"] * c["tokens"], "flops": 6 * n}
    if c["op"] == "conv":
        lens, width = _lens(c), c["width"] - 1
        rows = 2 * sum(lens) + sum(1 for x in lens if x) * width * (1 if c["fresh"] else 2)
        return {"bytes": rows * c["channels"] * size + 4 * c["channels"] * c["width"], "flops": 2 * sum(lens) * c["channels"] * c["width"]}
    live = c["batch"] - len(_empty(c))
    rows = live * c["q_len"]
    return {"bytes": live * c["v_heads"] * 65536 * (1 if c["fresh"] else 2)
            + rows * size * (2 * c["k_heads"] * 128 + 2 * c["v_heads"] * 128 + 2 * c["v_heads"]), "flops": 7 * rows * c["v_heads"] * 16384}


# ----------------------------------------------------------------- inputs

def _axis_of(c):
    """Which position axis turns each pair of a head's rotated dimensions: the pairs are dealt out in turn."""
    return [i % c["axes"] for i in range(c["rotary"] // 2)]


def _where(c):
    """Positions [axes, tokens] up to `far`: text, then an image whose rows and columns count from its start, then text."""
    n, far = c["tokens"], c["far"]
    at = torch.arange(n, device="cuda") * max(1, (far - 1) // n) if n * 8 <= far else far - 1 - torch.arange(n - 1, -1, -1, device="cuda") % far
    at = at.clamp(min=0)
    if c["axes"] == 1:
        return at[None].contiguous()
    side, a, b = 24, n // 4, n // 2
    grid = torch.arange(b - a, device="cuda")
    rows = torch.stack([at, at, at])
    if b > a:
        rows[0, a:b] = at[a]
        rows[1, a:b] = at[a] + grid // side % side
        rows[2, a:b] = at[a] + grid % side
    return rows


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = dict(c, dtype=dtype, work=None)
    if c["op"] == "quantize":
        loud = 1 + 40 * (uniform(c["cols"]) > 0.995)  # some channels are large
        s["x"] = (normal(c["rows"], c["cols"]) * loud).to(dtype)
        return s
    if c["op"] == "linear":
        loud = 1 + 40 * (uniform(c["k"]) > 0.995)
        s["x"] = (normal(c["m"], c["k"]) * loud).to(dtype)
        # the weight as a checkpoint holds it: codes, and a scale for each block
        codes, scales = _quantized(normal(c["n"], c["k"]) * 0.02, 128)
        s["codes"], s["scales"] = codes.view(torch.uint8), scales
        return s
    if c["op"] == "rope":
        dim, width = c["dim"], (c["q_heads"] + c["k_heads"]) * c["dim"]
        x = normal(c["tokens"], width + c["k_heads"] * dim)  # queries, keys and values side by side, as one projection gives them
        x = (x * (0.5 + 2 * uniform(1, x.shape[1]))).to(dtype)
        s["q"], s["k"] = x[:, : c["q_heads"] * dim], x[:, c["q_heads"] * dim: width]
        s["positions"] = _where(c)
        s["axis"] = torch.tensor(_axis_of(c), dtype=torch.uint8, device="cuda")
        half = c["rotary"] // 2
        s["freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        s["qw"], s["kw"] = ((0.2 * normal(dim) + (0.0 if c["offset"] else 1.0)) if c["norm"] else None for _ in range(2))
        return s
    if c["op"] == "conv":
        lens, ch, size = _lens(c), c["channels"], c["width"] - 1
        total = sum(lens)
        x = normal(total + 3, ch + 8 * (ch // 16))  # a part of a wider projection's columns, rows to spare behind the last sequence
        s["x"] = x.to(dtype)[:, :ch]
        s["weight"] = 0.5 * normal(ch, c["width"])
        s["b"] = 0.2 * normal(ch) if c["bias"] else None
        slots = torch.randperm(c["seqs"] + 3, generator=gen, device="cuda")[: c["seqs"]].int()
        if c["seqs"] > 1 and c["longest"] == 1:
            slots[c["seqs"] // 2] = -1  # a place of a padded batch: no state
        s["slots"] = slots
        s["state"] = normal(c["seqs"] + 3, size, ch).to(dtype)
        s["starts"] = None if c["longest"] == 1 else torch.tensor([0] + lens, device="cuda").cumsum(0).int()
        s["first"] = (torch.arange(c["seqs"], device="cuda") % 2).to(torch.uint8) if c["fresh"] else None  # half the sequences begin
        if c["longest"] == 1:
            s["x"] = s["x"][:total]
        # rows behind the last sequence are not the operator's: both sides start from the same ones
        s["y"] = torch.zeros(len(s["x"]), ch, dtype=dtype, device="cuda")
        return s
    rows, hk, hv = c["batch"] * c["q_len"], c["k_heads"], c["v_heads"]
    x = normal(rows, (2 * hk + hv) * 128).to(dtype)  # what the convolution gives: queries, keys, values
    s["q"], s["k"], s["v"] = x[:, : hk * 128], x[:, hk * 128: 2 * hk * 128], x[:, 2 * hk * 128:]
    s["beta"] = torch.sigmoid(normal(rows, hv)).to(dtype)
    s["g"] = (-(1 + 15 * uniform(hv)) * torch.nn.functional.softplus(0.5 * normal(rows, hv) - 5)).to(dtype)
    slots = torch.randperm(c["batch"] + 2, generator=gen, device="cuda")[: c["batch"]].int()
    for b in _empty(c):
        slots[b] = -1
    s["slots"] = slots
    s["states"] = 0.1 * normal(c["batch"] + 2, hv, 128, 128)
    s["first"] = (torch.arange(c["batch"], device="cuda") % 2).to(torch.uint8) if c["fresh"] else None
    s["o"] = torch.zeros(rows, hv * 128, dtype=dtype, device="cuda")
    return s


# -------------------------------------------------------------- one pass

def _blocks(x, block):
    """x [rows, cols] padded with zeros to whole blocks, as [row blocks, block, column blocks, 128]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % block))
    return x.view(-1, block, x.shape[1] // 128, 128)


def _quantized(x, block):
    """E4M3 codes of x and the scales of its blocks: scale = max / 448 in float32, a code the nearest to x / scale, ties to even. Both
    quotients are formed in 64 bits: 32 would put some next to a border on the wrong side."""
    rows, cols = x.shape
    b = _blocks(x.float(), block)
    scale = (b.abs().amax(dim=(1, 3)).double() / 448.0).float()
    y = b.double() / scale.double().clamp(min=1e-60)[:, None, :, None]
    step = (torch.frexp(y).exponent.clamp(min=-5).long() + (1023 - 4) << 52).view(torch.float64)  # the power of two itself
    y = (torch.round(y / step) * step).clamp(-448, 448).view(b.shape[0] * block, -1)[:rows, :cols]
    return y.to(torch.float8_e4m3fn), scale


def _dense(codes, scale, block):
    rows, cols = codes.shape
    return (_blocks(codes.float(), block) * scale[:, None, :, None]).view(-1, scale.shape[1] * 128)[:rows, :cols]


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "quantize":
        return _quantized(s["x"], s["block"])
    if s["op"] == "linear":
        x = _dense(*_quantized(s["x"], 1), 1)
        w = _dense(s["codes"].view(torch.float8_e4m3fn), s["scales"], 128)
        return torch.matmul(x, w.t()).to(s["dtype"])
    if s["op"] == "rope":
        turn = s["positions"].double()[s["axis"].long()] * s["freq"].double()[:, None]  # angles of far positions need 64 bits
        cos, sin = torch.cos(turn).float().t()[:, None], torch.sin(turn).float().t()[:, None]  # [tokens, 1, pairs]
        return tuple(_turned(s, x, w, cos, sin) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    if s["op"] == "conv":
        return _conv(s)
    return _step(s)


def _turned(s, x, w, cos, sin):
    x = x.float().reshape(s["tokens"], -1, s["dim"])
    if s["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (w + 1.0 if s["offset"] else w)
    r, half = s["rotary"], s["rotary"] // 2
    if s["pairs"] == "half":
        a, b = x[..., :half], x[..., half:r]
        parts = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        parts = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).reshape(len(x), -1, r)
    return torch.cat([parts, x[..., r:]], -1).reshape(len(x), -1).to(s["dtype"])


def _conv(s):
    size, seqs, device = s["width"] - 1, s["seqs"], s["x"].device
    starts = torch.arange(seqs + 1, device=device) if s["starts"] is None else s["starts"].long()
    total, lens = int(s["y"].shape[0] - (0 if s["starts"] is None else 3)), starts[1:] - starts[:-1]
    # the inputs that each sequence has before its first token
    kept = (s["slots"] >= 0) if s["first"] is None else (s["slots"] >= 0) & (s["first"] == 0)
    past = s["state"][s["slots"].clamp(min=0).long()].float() * kept[:, None, None]
    x = s["x"][:total].float()
    at = torch.arange(total, device=device)
    of = torch.searchsorted(starts, at, right=True) - 1  # the token's sequence
    since = at - starts[of]
    y = (torch.zeros_like(x) if s["b"] is None else s["b"].expand_as(x).clone())
    for j in range(s["width"]):  # the tap for the input `back` tokens ago
        back = size - j
        before = x.roll(back, 0)
        old = (since < back).nonzero()[:, 0]
        if back:
            before[old] = past[of[old], size - back + since[old]]
        y += before * s["weight"][:, j]
    if s["silu"]:
        y = y * torch.sigmoid(y)
    s["y"][:total] = y.to(s["dtype"])
    # the last inputs of each sequence, its old ones among them where it is short, are kept for its next call
    live = ((s["slots"] >= 0) & (lens > 0)).nonzero()[:, 0]
    back = torch.arange(size, device=device)[None] - size + lens[live][:, None]  # token of the sequence, negative: an old input
    new = x[(starts[live][:, None] + back).clamp(min=0)]
    old = torch.gather(past[live], 1, (back + size).clamp(0, size - 1)[:, :, None].expand(-1, -1, x.shape[1]))
    s["state"][s["slots"][live].long()] = torch.where((back >= 0)[:, :, None], new, old).to(s["dtype"])
    return s["y"], s["state"]


def _step(s):
    n, hk, hv = s["q_len"], s["k_heads"], s["v_heads"]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][live].long()

    def heads(x, h):
        return x.float().reshape(s["batch"], n, h, -1)[live]

    q, k = (x / x.norm(dim=-1, keepdim=True).clamp(min=1e-30) for x in (heads(s["q"], hk), heads(s["k"], hk)))
    q, k = ((x * f).repeat_interleave(hv // hk, 2) for x, f in ((q, 128 ** -0.5), (k, 1.0)))
    v, beta, g = heads(s["v"], hv), heads(s["beta"], hv), heads(s["g"], hv)
    state = s["states"][slots]
    if s["first"] is not None:
        state = state * (s["first"][live] == 0)[:, None, None, None]
    out = []
    for t in range(n):
        state = state * torch.exp(g[:, t])[..., None]
        u = beta[:, t] * (v[:, t] - (state * k[:, t, :, None, :]).sum(-1))
        state = state + u[..., None] * k[:, t, :, None, :]
        out.append((state * q[:, t, :, None, :]).sum(-1))
    s["states"][slots] = state
    o = s["o"].view(s["batch"], n, -1)
    o[live] = torch.stack(out, 1).reshape(len(live), n, -1).to(s["dtype"])
    return s["o"], s["states"]


def _own(s):
    import bit_linear_layer_amd as nv

    if s["op"] == "quantize":
        q = nv.fp8_quantize(s["x"], block_rows=s["block"])
        return q.codes[:, : s["cols"]].view(torch.float8_e4m3fn), q.scales[:, : -(-s["cols"] // 128)]
    if s["op"] == "linear":
        if s["work"] is None:  # a server keeps its weight's description and its workspace
            w = nv.FP8Tensor(s["codes"], s["scales"], s["n"], s["k"], 128)
            s["work"] = w, nv.fp8_linear_workspace(s["m"], s["k"], s["x"].device)
        w, space = s["work"]
        return nv.fp8_linear(s["x"], w, out_dtype=s["dtype"], workspace=space)
    if s["op"] == "rope":
        if s["work"] is None:
            s["work"] = nv.Rope(s["freq"], s["axis"] if s["axes"] > 1 else None, interleaved=s["pairs"] == "next")
        return nv.qk_norm_rope(s["q"], s["k"], s["dim"], s["positions"], s["work"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                               weight_offset=1.0 if s["offset"] else 0.0)
    if s["op"] == "conv":
        nv.nvfp4_causal_conv(s["x"], s["weight"], s["y"], s["seqs"], starts=s["starts"], bias=s["b"], silu=s["silu"],
                             state=s["state"], slots=s["slots"], fresh=s["first"])
        return s["y"], s["state"]
    nv.nvfp4_gdn_step(s["q"], s["k"], s["v"], s["beta"], s["g"], s["o"], s["k_heads"], s["v_heads"], s["states"], s["slots"],
                      q_len=s["q_len"], fresh=s["first"])
    return s["o"], s["states"]


# ------------------------------------------------------ the definition, in 64 bits

def _scales_64(x, block):
    """float32 scales, as 64-bit numbers, of the blocks of x (64 bits)."""
    rows, cols = x.shape
    out = torch.zeros(-(-rows // block), -(-cols // 128), dtype=torch.float64, device=x.device)
    for j in range(out.shape[1]):
        top = x[:, j * 128: (j + 1) * 128].abs().amax(1)
        if block > 1:
            top = torch.stack([part.amax() for part in top.split(block)])
        out[:, j] = (top / 448.0).float().double()
    return out


def _nearest_64(x, scales, block):
    """The E4M3 value nearest to x / scale, times the scale's place: [rows, cols] of values without the scale."""
    out = torch.empty_like(x)
    for j in range(scales.shape[1]):
        s = scales[:, j].repeat_interleave(block)[: len(x), None]
        y = torch.where(s > 0, x[:, j * 128: (j + 1) * 128] / s, 0.0)
        lead = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20)))
        lead = torch.where(y.abs() < torch.exp2(lead), lead - 1, torch.where(y.abs() >= torch.exp2(lead + 1), lead + 1, lead))
        grid = torch.exp2(lead.clamp(min=-6) - 3)
        out[:, j * 128: (j + 1) * 128] = (torch.round(y / grid) * grid).clamp(-448, 448)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        x = s["x"].double()
        scales = _scales_64(x, s["block"])
        return _nearest_64(x, scales, s["block"]), scales
    if s["op"] == "linear":
        x = s["x"].double()
        scales = _scales_64(x, 1)
        x = _nearest_64(x, scales, 1)
        table = []
        for b in range(256):
            e, m = b >> 3 & 15, b & 7
            mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            table.append(-mag if b & 128 else mag)
        w = torch.tensor(table, dtype=torch.float64, device="cuda")[s["codes"].int()]
        for j in range(scales.shape[1]):
            at = slice(j * 128, (j + 1) * 128)
            x[:, at] *= scales[:, j, None]
            w[:, at] *= s["scales"][:, j].double().repeat_interleave(128)[: len(w), None]
        return torch.mm(x, w.t())
    if s["op"] == "rope":
        out = []
        half, r, at = s["rotary"] // 2, s["rotary"], s["positions"].double()
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.double().reshape(s["tokens"], -1, s["dim"]).clone()
            if s["norm"]:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * (w.double() + (1.0 if s["offset"] else 0.0))
            for i, axis in enumerate(_axis_of(case)):
                a, b = (i, i + half) if s["pairs"] == "half" else (2 * i, 2 * i + 1)
                turn = (at[axis] * s["freq"][i].double())[:, None]
                u, v = x[:, :, a].clone(), x[:, :, b].clone()
                x[:, :, a], x[:, :, b] = u * torch.cos(turn) - v * torch.sin(turn), u * torch.sin(turn) + v * torch.cos(turn)
            out.append(x.reshape(len(x), -1))
        return tuple(out)
    if s["op"] == "conv":
        size, y, state = s["width"] - 1, s["y"].double(), s["state"].double()
        at = 0
        for b, n in enumerate(_lens(case)):
            slot = int(s["slots"][b])
            old = torch.zeros(size, s["channels"], dtype=torch.float64, device="cuda")
            if slot >= 0 and (s["first"] is None or not int(s["first"][b])):
                old = s["state"][slot].double()
            line = torch.cat([old, s["x"][at: at + n].double()])
            z = sum(line[j: j + n] * s["weight"][:, j].double() for j in range(s["width"]))
            z = z if s["b"] is None else z + s["b"].double()
            y[at: at + n] = z / (1 + torch.exp(-z)) if s["silu"] else z
            if slot >= 0 and n:
                state[slot] = line[n:]
            at += n
        return y, state
    n, hk, hv = s["q_len"], s["k_heads"], s["v_heads"]
    o, states = s["o"].double(), s["states"].double()
    eye = torch.eye(128, dtype=torch.float64, device="cuda")
    for b in range(s["batch"]):
        slot = int(s["slots"][b])
        if slot < 0:
            continue
        S = states[slot]
        if s["first"] is not None and int(s["first"][b]):
            S = torch.zeros_like(S)
        for t in range(b * n, b * n + n):
            q, k = (s[x][t].double().view(hk, 1, 128).expand(hk, hv // hk, 128).reshape(hv, 128, 1) for x in ("q", "k"))
            q, k = q / q.square().sum(1, keepdim=True).sqrt() * 128 ** -0.5, k / k.square().sum(1, keepdim=True).sqrt()
            beta, v = s["beta"][t].double().view(hv, 1, 1), s["v"][t].double().view(hv, 128, 1)
            kt = k.transpose(1, 2).contiguous()
            S = torch.exp(s["g"][t].double()).view(hv, 1, 1) * torch.bmm(S, eye - beta * k * kt) + beta * v * kt
            o[t] = torch.bmm(S, q).view(-1)
        states[slot] = S
    return o, states
