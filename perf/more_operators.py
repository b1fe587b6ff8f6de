"""Measured cases of the layer operators of a gated feed-forward sublayer: the gated linear layer, dropout from a
counter-based generator, and the residual sum with the norms around it, each forward and backward.

``run`` is the plain form (fp32 torch operations, rounded once at the end) or, with ``own`` set, the calls a
user makes of ``communication_compressed_optimizer_compress_gb300.layers``.

Shapes: hidden 1024, feed-forward 4096 and sequences of 512 tokens are those of the BERT-Large parameter
list that this repository's workloads use; the other sizes are generic.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 64            # columns that share one scale of an 8-bit checkpoint
TINY = 2.0 ** -120    # a block whose largest magnitude is below this is held as zeros
EPS = 1e-5


def listed():
    return [
        # a single token through the gated layer, as a step of generation meets it: the weights' bytes and latency
        dict(name="gated_fwd_1x1024x4096_bf16", op="gated_fwd", rows=1, k=1024, n=4096, dtype="bf16", pad=0, act="silu",
             bias=False, keep="none"),
        # a micro-batch of 32 sequences of 512 tokens in training, gate and up values kept in 16 bits
        dict(name="gated_fwd_16384x1024x4096_bf16", op="gated_fwd", rows=16384, k=1024, n=4096, dtype="bf16", pad=0,
             act="silu", bias=False, keep="values"),
        # odd sizes in every direction, a packed batch of 777 tokens with 8-bit checkpoints, rows that start at any 2-byte boundary
        dict(name="gated_fwd_777x1001x1155_f16_ck", op="gated_fwd", rows=777, k=1001, n=1155, dtype="f16", pad=2,
             act="gelu_tanh", bias=True, keep="checkpoint"),
        # the backward pass of the training micro-batch from 8-bit checkpoints: through the second product to gate and up
        dict(name="gated_bwd_16384x4096x1024_bf16_ck", op="gated_bwd", rows=16384, n=4096, out=1024, dtype="bf16", pad=0,
             act="silu", keep="checkpoint", grad="bf16"),
        # the backward pass of one short odd sequence from 16-bit values
        dict(name="gated_bwd_333x1030x520_f16", op="gated_bwd", rows=333, n=1030, out=520, dtype="f16", pad=0, act="gelu",
             keep="values", grad="f16"),
        # dropout of a micro-batch's feed-forward activations
        dict(name="dropout_16384x4096_bf16", op="dropout", rows=16384, cols=4096, dtype="bf16", pad=0, p=0.1),
        # odd rows and columns out of a wider fp32 buffer (no row is aligned)
        dict(name="dropout_4099x1155_f32", op="dropout", rows=4099, cols=1155, dtype="f32", pad=6, p=0.5),
        # 16 single tokens between two blocks of a model with norms behind and before its blocks: latency alone
        dict(name="rn_fwd_16x1024_bf16_rms", op="rn_fwd", rows=16, cols=1024, dtype="bf16", pad=0, norm="rms", post=True,
             gate=True, scale=1.0, p=0.0),
        # a micro-batch in training as BERT has it: dropout of the block's output, residual sum, layer norm
        dict(name="rn_fwd_16384x1024_bf16", op="rn_fwd", rows=16384, cols=1024, dtype="bf16", pad=0, norm="layer",
             post=False, gate=False, scale=1.0, p=0.1),
        # its backward pass, with the gradient that the residual path brings
        dict(name="rn_bwd_16384x1024_bf16", op="rn_bwd", rows=16384, cols=1024, dtype="bf16", pad=0, norm="layer",
             post=False, gate=False, scale=1.0, p=0.1, grad="f32"),
        # the backward pass of RMS norms behind and before the block with a gate and a residual scale, fp16 gradients
        dict(name="rn_bwd_8192x2048_f16_rms", op="rn_bwd", rows=8192, cols=2048, dtype="f16", pad=0, norm="rms", post=True,
             gate=True, scale=0.5, p=0.1, grad="f16"),
        # odd rows and columns out of a wider buffer, every option at once
        dict(name="rn_bwd_1237x1001_bf16", op="rn_bwd", rows=1237, cols=1001, dtype="bf16", pad=3, norm="layer", post=True,
             gate=True, scale=0.5, p=0.1, grad="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ranges: 1 to 16384 rows and widths 32 to 4096 for the products, 1 to 65536 rows and widths 16 to
    8192 for the row operators, at most the largest listed case's work."""
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "dropout", "rn_fwd", "rn_fwd", "rn_bwd", "rn_bwd"])
    dtype = rng.choice(["bf16", "f16"] if op.startswith("gated") else ["bf16", "f16", "f32"])
    pad = rng.choice([0, 0, 0, 1, 8, 24])
    case = dict(op=op, dtype=dtype, pad=pad)
    if op.startswith("gated"):
        a, n = _log(rng, 32, 4096), _log(rng, 32, 4096)
        if rng.random() < 0.6:
            a, n = max(32, a // 32 * 32), max(32, n // 32 * 32)
        case["rows"] = max(1, min(_log(rng, 1, 16384), 16384 * 1024 * 4096 // (a * n)))
        case.update(n=n, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu", "none"]))
        if op == "gated_fwd":
            case.update(k=a, bias=rng.random() < 0.5, keep=rng.choice(["none", "values", "checkpoint"]))
        else:
            case.update(out=a, keep=rng.choice(["values", "checkpoint"]), grad=dtype)
        return case
    cols = _log(rng, 16, 8192)
    if rng.random() < 0.5:
        cols = max(16, cols // 64 * 64)
    case["rows"] = min(_log(rng, 1, 65536), (1 << 25) // cols)
    case["cols"] = cols
    case["p"] = rng.choice([0.0, 0.1, 0.5, round(rng.uniform(0.01, 0.9), 3)])
    if op == "dropout":
        case["p"] = max(case["p"], 0.1)
        return case
    case.update(norm=rng.choice(["layer", "rms"]), post=rng.random() < 0.5, gate=rng.random() < 0.5, scale=rng.choice([1.0, 0.5, 0.125]))
    if op == "rn_bwd":
        case["grad"] = rng.choice(["f32", dtype])
    return case


# ---------------------------------------------------------------- inputs


def _rows(t, pad):
    """The same values as the left columns of a buffer that is `pad` columns wider."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def _activation(gen, rows, cols, dtype):
    """Activations: a small mean and, as in trained networks, a few columns of larger magnitude."""
    x = torch.randn(rows, cols, generator=gen, device="cuda") + 0.1
    x *= torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.01, 6.0, 1.0)
    return x.to(dtype)


def _quantise(x):
    """Codes and scales of an 8-bit checkpoint, in fp32: blocks of 64 columns of a row."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.zeros(rows, blocks * BLOCK, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, blocks, BLOCK)
    most = v.abs().amax(2)
    zero = most < TINY
    scales = torch.where(zero, 0.0, most / 127)
    codes = torch.round(v * torch.where(zero, 0.0, 127 / most)[:, :, None])
    return codes.to(torch.int8).view(rows, blocks * BLOCK)[:, :cols].contiguous(), scales


def _values(codes, scales):
    return codes.float() * scales.repeat_interleave(BLOCK, 1)[:, : codes.shape[1]]


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    rows, dtype, op, pad = case["rows"], DTYPES[case["dtype"]], case["op"], case["pad"]
    s = dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if op == "gated_fwd":
        k, n = case["k"], case["n"]
        s["x"] = _rows((randn(rows, k) + 0.1).to(dtype), pad)
        s["w"] = (randn(2 * n, k) * (1.5 / math.sqrt(k))).to(dtype)
        s["b"] = 0.1 * randn(2 * n) if case["bias"] else None
        return s
    if op == "gated_bwd":
        n, out = case["n"], case["out"]
        z = (1.5 * randn(rows, 2 * n) + 0.1).to(dtype)
        if case["keep"] == "checkpoint":
            s["gate_codes"], s["gate_scales"] = _quantise(z[:, :n])
            s["up_codes"], s["up_scales"] = _quantise(z[:, n:])
        else:
            s["z"] = _rows(z, pad)
        s["w"] = (randn(out, n) * (1 / math.sqrt(n))).to(dtype)
        s["dy"] = _rows((0.05 * randn(rows, out)).to(dtype), pad)
        return s
    # the seed of the masks and the number of the training step
    s["key"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")
    s["site"] = 3
    cols = case["cols"]
    x = _activation(gen, rows, cols, dtype)
    if op == "dropout":
        s["x"] = _rows(x, pad)
        return s
    layer = case["norm"] == "layer"
    block = (0.5 * randn(rows, cols) + 0.05).to(dtype)
    s["block"] = _rows(block, pad)
    s["gamma"] = 1 + 0.1 * randn(cols)
    s["beta"] = 0.1 * randn(cols) if layer else None
    s["block_gamma"] = 1 + 0.1 * randn(cols) if case["post"] else None
    s["block_beta"] = 0.1 * randn(cols) if case["post"] and layer else None
    s["gatev"] = 0.5 + 0.1 * randn(cols) if case["gate"] else None
    s["x"] = _rows(x, pad)
    if op == "rn_bwd":
        # what the forward pass leaves
        f = _rn_forward(s)
        del s["x"]
        s["s"] = _rows(f["s"].to(dtype), pad)
        s.update({name: f[name] for name in ("mean", "rstd", "block_mean", "block_rstd")})
        s["dy"] = _rows((0.05 * randn(rows, cols)).to(dtype), pad)
        s["ds"] = _rows((0.05 * randn(rows, cols)).to(dtype), pad)
    return s


# ---------------------------------------------------------------- the plain form


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(name, z):
    if name == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q + z * q * (1 - q)
    if name == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * (math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z))
    return torch.ones_like(z)


def _mask(rows, cols, p, key, site):
    """Which elements stay, and the factor on them: Philox4x32-10 of the group of eight columns, 16 bits an element."""
    groups = -(-cols // 8)
    threshold = round(p * 65536)
    low = 0xFFFFFFFF
    i = torch.arange(rows * groups, device=key.device)
    step = (key[1] & low).expand_as(i)
    c = [i & low, i >> 32, step, torch.full_like(i, site)]
    k = [key[0] & low, (key[0] >> 32) & low]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]  # the products' 64 bits, whatever their sign
        c = [((b >> 32) & low) ^ c[1] ^ k[0], b & low, ((a >> 32) & low) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    bits = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 1).view(rows, groups * 8)[:, :cols]
    return bits >= threshold, 65536 / (65536 - threshold)


def _norm(v, layer):
    mean = v.mean(1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
    rstd = 1 / torch.sqrt((v - mean).square().mean(1, keepdim=True) + EPS)
    return (v - mean) * rstd, mean, rstd


def _rn_forward(s):
    layer = s["norm"] == "layer"
    n = s["block"].float()
    got = dict(block_mean=None, block_rstd=None)
    if s["post"]:
        n, mean, rstd = _norm(n, layer)
        n = n * s["block_gamma"]
        if layer:
            n = n + s["block_beta"]
        got.update(block_mean=mean[:, 0] if layer else None, block_rstd=rstd[:, 0])
    if s["p"] > 0:
        stays, factor = _mask(*n.shape, s["p"], s["key"], s["site"])
        n = torch.where(stays, n * factor, 0.0)
    if s["gate"]:
        n = n * s["gatev"]
    got["s"] = s["x"].float() + s["scale"] * n
    y, mean, rstd = _norm(got["s"], layer)
    y = y * s["gamma"]
    got.update(y=y + s["beta"] if layer else y, mean=mean[:, 0] if layer else None, rstd=rstd[:, 0])
    return got


def _norm_grad(g, xhat, rstd, layer):
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if layer:
        d = d - g.mean(1, keepdim=True)
    return d * rstd[:, None]


def _rn_backward(s):
    layer, grad, dtype = s["norm"] == "layer", DTYPES[s["grad"]], DTYPES[s["dtype"]]
    dy, block = s["dy"].float(), s["block"].float()
    xhat = s["s"].float()
    if layer:
        xhat = xhat - s["mean"][:, None]
    xhat = xhat * s["rstd"][:, None]
    t = _norm_grad(dy * s["gamma"], xhat, s["rstd"], layer) + s["ds"].float()
    d = s["scale"] * t
    if s["p"] > 0:
        stays, factor = _mask(*t.shape, s["p"], s["key"], s["site"])
        d = torch.where(stays, d * factor, 0.0)
    out = [t.to(dtype), None, (dy * xhat).sum(0).to(grad)] + ([dy.sum(0).to(grad)] if layer else [])
    dn = d * s["gatev"] if s["gate"] else d
    n = block
    if s["post"]:
        bhat = block - s["block_mean"][:, None] if layer else block
        bhat = bhat * s["block_rstd"][:, None]
        n = bhat * s["block_gamma"]
        if layer:
            n = n + s["block_beta"]
        out.append((dn * bhat).sum(0).to(grad))
        if layer:
            out.append(dn.sum(0).to(grad))
        dn = _norm_grad(dn * s["block_gamma"], bhat, s["block_rstd"], layer)
    if s["gate"]:
        out.append((d * n).sum(0).to(grad))
    out[1] = dn.to(dtype)
    return out


def _plain(s):
    op, dtype = s["op"], DTYPES[s["dtype"]]
    if op == "gated_fwd":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"]
        g, u = z[:, : s["n"]], z[:, s["n"]:]
        h = (_act(s["act"], g) * u).to(dtype)
        if s["keep"] == "none":
            return [h]
        return [h, z.to(dtype)] if s["keep"] == "values" else [h, _values(*_quantise(g)).to(dtype), _values(*_quantise(u)).to(dtype)]
    if op == "gated_bwd":
        if s["keep"] == "checkpoint":
            g, u = _values(s["gate_codes"], s["gate_scales"]), _values(s["up_codes"], s["up_scales"])
        else:
            g, u = s["z"][:, : s["n"]].float(), s["z"][:, s["n"]:].float()
        dy = s["dy"].float()
        dh = dy @ s["w"].float()
        a = _act(s["act"], g)
        dz = torch.cat([dh * u * _act_grad(s["act"], g), dh * a], 1)
        grad = DTYPES[s["grad"]]
        return [dz.to(dtype), (dy.t() @ (a * u)).to(grad), dy.sum(0).to(grad)]
    if op == "dropout":
        stays, factor = _mask(*s["x"].shape, s["p"], s["key"], s["site"])
        return torch.where(stays, s["x"].float() * factor, 0.0).to(dtype)
    if op == "rn_bwd":
        return _rn_backward(s)
    f = _rn_forward(s)
    out = [f["y"].to(dtype), f["s"].to(dtype)]
    return out + [f[name] for name in ("mean", "rstd", "block_mean", "block_rstd") if f[name] is not None]


def _own(s):
    from communication_compressed_optimizer_compress_gb300 import layers

    op, dtype = s["op"], DTYPES[s["dtype"]]
    if op == "dropout":
        return layers.dropout(s["x"], s["p"], s["key"], s["site"])
    if op.startswith("gated"):
        act = layers.GATE_ACTIVATIONS[s["act"]]
        if op == "gated_bwd":
            if s["keep"] == "checkpoint":
                z = layers.Gated(layers.Checkpoint(s["gate_codes"], s["gate_scales"], dtype),
                                 layers.Checkpoint(s["up_codes"], s["up_scales"], dtype))
            else:
                z = s["z"]
            return layers.gated_linear_backward(s["dy"], z, s["w"], act, grad_dtype=DTYPES[s["grad"]])
        if s["keep"] == "none":
            return [layers.gated_linear(s["x"], s["w"], s["b"], act)]
        h, z = layers.gated_linear(s["x"], s["w"], s["b"], act, keep=s["keep"])
        return [h, z] if s["keep"] == "values" else [h, layers.restore(z.gate), layers.restore(z.up)]
    options = dict(norm=layers.NORMS[s["norm"]], block_gamma=s["block_gamma"], block_beta=s["block_beta"], gate=s["gatev"],
                   scale=s["scale"], p=s["p"], key=s["key"], site=s["site"])
    if op == "rn_fwd":
        r = layers.residual_norm(s["x"], s["block"], s["gamma"], s["beta"], EPS, **options)
        got = [r.y, r.s, r.mean, r.rstd, r.block_mean, r.block_rstd]
    else:
        got = layers.residual_norm_backward(s["dy"], s["ds"], s["s"], s["block"], s["gamma"], s["mean"], s["rstd"],
                                            block_mean=s["block_mean"], block_rstd=s["block_rstd"],
                                            grad_dtype=DTYPES[s["grad"]], **options)
    return [t for t in got if t is not None]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass needs


def work(case):
    rows, e, op = case["rows"], BYTES[case["dtype"]], case["op"]
    if op.startswith("gated"):
        n = case["n"]
        kept = {"none": 0, "values": 2 * e * rows * n, "checkpoint": 2 * rows * (n + 4 * -(-n // BLOCK))}[case["keep"]]
        if op == "gated_fwd":  # a checkpoint is read back too
            k = case["k"]
            back = kept + 2 * e * rows * n if case["keep"] == "checkpoint" else 0
            return {"bytes": e * (rows * k + 2 * n * k + rows * n) + (8 * n if case["bias"] else 0) + kept + back, "flops": 4 * rows * n * k}
        out = case["out"]
        return {"bytes": e * (rows * out + out * n + 2 * rows * n) + kept + BYTES[case["grad"]] * (out * n + out),
                "flops": 4 * rows * n * out}
    cols = case["cols"]
    full = rows * cols * e
    if op == "dropout":
        return {"bytes": 2 * full + 16, "flops": 12 * rows * cols}
    layer, post, gate = case["norm"] == "layer", case["post"], case["gate"]
    stats = 4 * rows * (1 + layer) * (1 + post)
    vectors = cols * ((1 + layer) * (1 + post) + gate)
    if op == "rn_fwd":
        return {"bytes": 4 * full + stats + 4 * vectors, "flops": 20 * rows * cols}
    block = full if post or gate else 0  # its values enter no gradient otherwise
    read = cols * (1 + (2 if layer else 1) * post + gate)
    return {"bytes": 5 * full + block + stats + 4 * read + BYTES[case["grad"]] * vectors, "flops": 30 * rows * cols}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_kept(x):
    """The values that an 8-bit checkpoint of x stands for, block by block of 64 columns."""
    got = []
    for piece in x.split(BLOCK, 1):
        most = piece.abs().max(1, keepdim=True).values
        step = most / 127
        got.append(torch.where(most < TINY, torch.zeros_like(piece), torch.round(piece / step) * step))
    return torch.cat(got, 1)


def _exact_act(name, z):
    """(activation, derivative) of z."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    u, du = (z / 2, 0.5) if name == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 0.134145 * z.square()))
    p = torch.sigmoid(2 * u)  # (1 + tanh u) / 2
    return z * p, p + z * 2 * p * (1 - p) * du


def _exact_factors(rows, cols, case, s):
    """What dropout multiplies each element with: the generator by halves of 16 bits, whose products and sums stay small."""
    if case["p"] <= 0:
        return torch.ones(rows, cols, dtype=torch.float64, device="cuda")
    seed, step = (int(v) for v in s["key"].tolist())

    def high_low(constant, v):
        """The upper and the lower 32 bits of constant * v."""
        ch, cl, vh, vl = constant // 65536, constant % 65536, v // 65536, v % 65536
        middle = ch * vl + cl * vh + cl * vl // 65536
        return ch * vh + middle // 65536, middle % 65536 * 65536 + cl * vl % 65536

    per = (cols + 7) // 8
    at = torch.arange(rows, device="cuda")[:, None] * per + torch.arange(per, device="cuda")[None, :]
    x0, x1 = at % 2 ** 32, at // 2 ** 32
    x2, x3 = torch.full_like(at, step % 2 ** 32), torch.full_like(at, s["site"])
    for r in range(10):
        k0, k1 = (seed + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        (h0, l0), (h1, l1) = high_low(0xD2511F53, x0), high_low(0xCD9E8D57, x2)
        x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
    factors = torch.empty(rows, per, 8, dtype=torch.float64, device="cuda")
    dropped = round(case["p"] * 65536)
    for e, word in enumerate((x0, x1, x2, x3)):
        factors[:, :, 2 * e] = (word % 65536 >= dropped).double()
        factors[:, :, 2 * e + 1] = (word // 65536 >= dropped).double()
    return factors.reshape(rows, per * 8)[:, :cols] * (65536 / (65536 - dropped))


def _exact_rn(case, s, d):
    layer, rows, cols = case["norm"] == "layer", case["rows"], case["cols"]
    through = _exact_factors(rows, cols, case, s) * case["scale"]
    if case["gate"]:
        through *= d["gatev"]

    def statistics(v):
        if layer:
            var, mean = torch.var_mean(v, 1, correction=0)
            return mean, (var + EPS) ** -0.5
        return None, (torch.linalg.vector_norm(v, dim=1).square() / cols + EPS) ** -0.5

    def standard(v, mean, rstd):
        return (v if mean is None else v - mean.unsqueeze(1)) * rstd.unsqueeze(1)

    def back(g, xh, rstd):
        along = torch.einsum("rc,rc->r", g, xh) / cols
        d = torch.addcmul(g, along.unsqueeze(1), xh, value=-1)
        return (d - g.sum(1, keepdim=True) / cols if layer else d) * rstd.unsqueeze(1)

    if case["op"] == "rn_fwd":
        n, tail = d["block"], []
        if case["post"]:
            bm, br = statistics(n)
            n = standard(n, bm, br) * d["block_gamma"]
            n = n + d["block_beta"] if layer else n
            tail = [bm, br] if layer else [br]
        total = torch.addcmul(d["x"], through, n)
        m, r = statistics(total)
        y = standard(total, m, r) * d["gamma"]
        return [y + d["beta"] if layer else y, total] + ([m, r] if layer else [r]) + tail
    xh = standard(d["s"], d.get("mean"), d["rstd"])
    t = back(d["dy"] * d["gamma"], xh, d["rstd"]) + d["ds"]
    out = [t, None, torch.einsum("rc,rc->c", d["dy"], xh)] + ([torch.einsum("rc->c", d["dy"])] if layer else [])
    dn, n = t * through, d["block"]
    if case["post"]:
        bh = standard(n, d.get("block_mean"), d["block_rstd"])
        out += [torch.einsum("rc,rc->c", dn, bh)] + ([torch.einsum("rc->c", dn)] if layer else [])
        n = bh * d["block_gamma"]
        n = n + d["block_beta"] if layer else n
        out[1] = back(dn * d["block_gamma"], bh, d["block_rstd"])
    else:
        out[1] = dn
    if case["gate"]:
        out.append(torch.einsum("rc,rc->c", t * _exact_factors(rows, cols, case, s), n) * case["scale"])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and k != "key"}
    if op == "dropout":
        factors = _exact_factors(case["rows"], case["cols"], case, s)
        return d["x"] * factors
    if op.startswith("rn"):
        return _exact_rn(case, s, d)
    n = case["n"]
    if op == "gated_fwd":
        g, u = (torch.mm(d["x"], w.mT) for w in d["w"].split(n))
        if case["bias"]:
            g, u = g + d["b"][:n], u + d["b"][n:]
        h = _exact_act(case["act"], g)[0] * u
        return [h] + {"none": [], "values": [torch.cat([g, u], 1)], "checkpoint": [_exact_kept(g), _exact_kept(u)]}[case["keep"]]
    if case["keep"] == "checkpoint":
        g, u = (torch.cat([c * d[name + "_scales"][:, i: i + 1] for i, c in enumerate(d[name + "_codes"].split(BLOCK, 1))], 1)
                for name in ("gate", "up"))
    else:
        g, u = d["z"].split(n, 1)
    a, slope = _exact_act(case["act"], g)
    dh = torch.mm(d["dy"], d["w"])
    return [torch.hstack([dh * slope * u, dh * a]), torch.mm(d["dy"].mT, a * u), torch.mv(d["dy"].mT, torch.ones_like(d["dy"][:, 0]))]
