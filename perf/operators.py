"""Measured cases of the layer operators: layer norm, the linear layer with its fused epilogue, and 8-bit
activation checkpoints, each forward and backward.

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
        # the normalisation of 16 single tokens, as a step of generation meets it: latency alone
        dict(name="ln_fwd_16x1024_bf16", op="ln_fwd", rows=16, cols=1024, dtype="bf16", pad=0, ckpt=False),
        # a micro-batch of 32 sequences of 512 tokens in training, its input kept in 8 bits for the backward pass
        dict(name="ln_fwd_16384x1024_bf16_ck", op="ln_fwd", rows=16384, cols=1024, dtype="bf16", pad=0, ckpt=True),
        # its backward pass from the 8-bit checkpoint, with the gradient that the residual path brings
        dict(name="ln_bwd_16384x1024_bf16_ck", op="ln_bwd", rows=16384, cols=1024, dtype="bf16", pad=0, ckpt=True,
             add=True, grad="f32"),
        # odd rows and columns out of a wider fp32 buffer (no row is aligned)
        dict(name="ln_bwd_4099x1155_f32", op="ln_bwd", rows=4099, cols=1155, dtype="f32", pad=6, ckpt=False, add=False,
             grad="f32"),
        # the feed-forward layer's first product for 16 tokens: the weight's bytes and latency
        dict(name="lin_fwd_16x1024x4096_bf16", op="lin_fwd", rows=16, k=1024, n=4096, dtype="bf16", pad=0, act="gelu",
             residual=False, ckpt=False),
        # the same product in training over 128 sequences of 512 tokens, the value before the gelu kept in 8 bits
        dict(name="lin_fwd_65536x1024x4096_ck", op="lin_fwd", rows=65536, k=1024, n=4096, dtype="bf16", pad=0,
             act="gelu", residual=False, ckpt=True),
        # the second product with its bias and the residual, in fp16 as the workload's gradients are
        dict(name="lin_fwd_16384x4096x1024_f16", op="lin_fwd", rows=16384, k=4096, n=1024, dtype="f16", pad=0,
             act="none", residual=True, ckpt=False),
        # odd sizes in every direction: a packed batch of 1237 tokens, rows that start at any 2-byte boundary
        dict(name="lin_fwd_1237x1001x777_bf16", op="lin_fwd", rows=1237, k=1001, n=777, dtype="bf16", pad=2,
             act="gelu_tanh", residual=True, ckpt=True),
        # the first product's backward pass: dx joined by the residual's gradient, fp32 dW and db
        dict(name="lin_bwd_16384x1024x4096_bf16", op="lin_bwd", rows=16384, k=1024, n=4096, dtype="bf16", pad=0,
             act="none", ckpt=False, add=True, grad="f32"),
        # the second product's backward pass through the gelu from the 8-bit checkpoint, fp16 gradients
        dict(name="lin_bwd_16384x4096x1024_ck", op="lin_bwd", rows=16384, k=4096, n=1024, dtype="f16", pad=0,
             act="gelu", ckpt=True, add=False, grad="f16"),
        # the backward pass of one short odd sequence
        dict(name="lin_bwd_333x520x1030_bf16", op="lin_bwd", rows=333, k=520, n=1030, dtype="bf16", pad=0, act="relu",
             ckpt=False, add=False, grad="bf16"),
        # the checkpoint by itself: a feed-forward activation held in 8 bits and read back
        dict(name="ck_16384x4096_bf16", op="ck", rows=16384, cols=4096, dtype="bf16", pad=0, act="none"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ranges: 1 to 65536 rows, widths 16 to 8192 for the row operators and 32 to 4096 for
    the products, at most the largest listed case's work."""
    op = rng.choice(["ln_fwd", "ln_bwd", "lin_fwd", "lin_fwd", "lin_bwd", "lin_bwd", "ck"])
    dtype = rng.choice(["bf16", "f16"] if op.startswith("lin") else ["bf16", "f16", "f32"])
    pad = rng.choice([0, 0, 0, 1, 8, 24])
    case = dict(op=op, rows=_log(rng, 1, 65536), dtype=dtype, pad=pad)
    if op in ("ln_fwd", "ln_bwd", "ck"):
        cols = _log(rng, 16, 8192)
        if rng.random() < 0.5:
            cols = max(16, cols // 64 * 64)
        case["rows"] = min(case["rows"], (1 << 28) // cols)
        case["cols"] = cols
        if op == "ck":
            case["act"] = rng.choice(["none", "gelu"])
        else:
            case["ckpt"] = rng.random() < 0.5
        if op == "ln_bwd":
            case.update(add=rng.random() < 0.5, grad=rng.choice(["f32", dtype]))
        return case
    k, n = _log(rng, 32, 4096), _log(rng, 32, 4096)
    if rng.random() < 0.6:
        k, n = max(32, k // 32 * 32), max(32, n // 32 * 32)
    most = 65536 * 1024 * 4096 // (2 if op == "lin_bwd" else 1)
    case["rows"] = max(1, min(case["rows"], most // (k * n)))
    case.update(k=k, n=n, act=rng.choice(["none", "relu", "gelu", "gelu_tanh"]), ckpt=rng.random() < 0.5)
    if op == "lin_fwd":
        case["residual"] = rng.random() < 0.5
    else:
        # a gradient that an activation rounded to 16 bits goes into is asked for in 16 bits
        case.update(add=rng.random() < 0.5, grad=dtype if case["ckpt"] or case["act"] != "none" else rng.choice(["f32", dtype]))
    return case


# ---------------------------------------------------------------- inputs


def _rows(t, pad):
    """The same values as the left columns of a buffer that is `pad` columns wider."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def _activation(gen, rows, cols, dtype, outliers=True):
    """Activations: a small mean and, as in trained networks, a few columns of larger magnitude."""
    x = torch.randn(rows, cols, generator=gen, device="cuda") + 0.1
    if outliers:
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

    if op in ("ln_fwd", "ln_bwd", "ck"):
        cols = case["cols"]
        x = _activation(gen, rows, cols, dtype)
        s["x"] = _rows(x, pad)
        if op == "ck":
            return s
        s["gamma"] = 1 + 0.1 * randn(cols)
        s["beta"] = 0.1 * randn(cols)
        if op == "ln_bwd":
            if case["ckpt"]:
                s["codes"], s["scales"] = _quantise(x)
                del s["x"]
            v = x.float()
            s["mean"] = v.mean(1)
            s["rstd"] = torch.rsqrt((v - s["mean"][:, None]).square().mean(1) + EPS)
            s["dy"] = _rows((0.05 * randn(rows, cols)).to(dtype), pad)
            s["add"] = (0.05 * randn(rows, cols)).to(dtype) if case["add"] else None
        return s
    k, n = case["k"], case["n"]
    s["w"] = (randn(n, k) * (1.5 / math.sqrt(k))).to(dtype)
    s["bias"] = 0.1 * randn(n)
    if op == "lin_fwd":
        s["x"] = _rows(_activation(gen, rows, k, dtype, outliers=False), pad)
        s["residual"] = _rows(_activation(gen, rows, n, dtype), pad) if case["residual"] else None
        return s
    x = _activation(gen, rows, k, dtype, outliers=False)
    if case["ckpt"]:
        s["codes"], s["scales"] = _quantise(x)
    else:
        s["x"] = _rows(x, pad)
    s["dy"] = _rows((0.05 * randn(rows, n)).to(dtype), pad)
    s["add"] = (0.05 * randn(rows, k)).to(dtype) if case["add"] else None
    return s


# ---------------------------------------------------------------- the plain form


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(name, z):
    if name == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * (math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z))


def _plain(s):
    op, dtype = s["op"], DTYPES[s["dtype"]]
    if op == "ck":
        return _act(s["act"], _values(*_quantise(s["x"].float()))).to(dtype)
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
        out = [((x - mean) * rstd * s["gamma"] + s["beta"]).to(dtype), mean[:, 0], rstd[:, 0]]
        if s["ckpt"]:
            out.append(_values(*_quantise(x)).to(dtype))
        return out
    if op == "ln_bwd":
        x = _values(s["codes"], s["scales"]) if s["ckpt"] else s["x"].float()
        dy = s["dy"].float()
        rstd = s["rstd"][:, None]
        xhat = (x - s["mean"][:, None]) * rstd
        g = dy * s["gamma"]
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        if s["add"] is not None:
            dx = dx + s["add"].float()
        grad = DTYPES[s["grad"]]
        return dx.to(dtype), (dy * xhat).sum(0).to(grad), dy.sum(0).to(grad)
    if op == "lin_fwd":
        z = s["x"].float() @ s["w"].float().t() + s["bias"]
        y = _act(s["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(dtype), _values(*_quantise(z)).to(dtype)] if s["ckpt"] else [y.to(dtype)]
    v = _values(s["codes"], s["scales"]) if s["ckpt"] else s["x"].float()
    dy = s["dy"].float()
    dx = dy @ s["w"].float()
    if s["act"] != "none":
        dx = dx * _act_grad(s["act"], v)
    if s["add"] is not None:
        dx = dx + s["add"].float()
    grad = DTYPES[s["grad"]]
    return dx.to(dtype), (dy.t() @ _act(s["act"], v)).to(grad), dy.sum(0).to(grad)


def _own(s):
    from communication_compressed_optimizer_compress_gb300 import layers

    op, dtype = s["op"], DTYPES[s["dtype"]]
    act = layers.ACTIVATIONS[s.get("act", "none")]
    if op == "ck":
        return layers.restore(layers.compress(s["x"]), activation=act)
    if op == "ln_fwd":
        if not s["ckpt"]:
            return layers.layer_norm(s["x"], s["gamma"], s["beta"], EPS)
        y, mean, rstd, ck = layers.layer_norm(s["x"], s["gamma"], s["beta"], EPS, checkpoint=True)
        return y, mean, rstd, layers.restore(ck)
    kept = layers.Checkpoint(s["codes"], s["scales"], dtype) if op.endswith("bwd") and s["ckpt"] else s["x"]
    if op == "ln_bwd":
        return layers.layer_norm_backward(s["dy"], kept, s["gamma"], s["mean"], s["rstd"], add=s["add"],
                                          grad_dtype=DTYPES[s["grad"]])
    if op == "lin_fwd":
        if not s["ckpt"]:
            return [layers.linear(s["x"], s["w"], s["bias"], act, s["residual"])]
        y, ck = layers.linear(s["x"], s["w"], s["bias"], act, s["residual"], checkpoint=True)
        return y, layers.restore(ck)
    return layers.linear_backward(s["dy"], kept, s["w"], act, add=s["add"], grad_dtype=DTYPES[s["grad"]])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass needs


def work(case):
    rows, e, op = case["rows"], BYTES[case["dtype"]], case["op"]
    if op in ("ln_fwd", "ln_bwd", "ck"):
        cols = case["cols"]
        kept = rows * cols + 4 * rows * -(-cols // BLOCK)  # codes and scales
        full = rows * cols * e
        if op == "ck":  # held in 8 bits, and read back
            return {"bytes": 2 * full + 2 * kept, "flops": 4 * rows * cols}
        if op == "ln_fwd":  # with the checkpoint it is read back too
            return {"bytes": 2 * full + 8 * rows + 8 * cols + (2 * kept + full if case["ckpt"] else 0),
                    "flops": 8 * rows * cols}
        return {"bytes": 2 * full + (kept if case["ckpt"] else full) + (full if case["add"] else 0) + 8 * rows + 4 * cols
                + 2 * BYTES[case["grad"]] * cols, "flops": 14 * rows * cols}
    k, n = case["k"], case["n"]
    if op == "lin_fwd":
        kept = rows * n + 4 * rows * -(-n // BLOCK)
        return {"bytes": e * (rows * k + n * k + rows * n * (2 if case["residual"] else 1)) + 4 * n
                + (2 * kept + e * rows * n if case["ckpt"] else 0), "flops": 2 * rows * n * k}
    kept = rows * k + 4 * rows * -(-k // BLOCK) if case["ckpt"] else rows * k * e
    return {"bytes": e * (rows * n + n * k + rows * k * (2 if case["add"] else 1)) + kept
            + BYTES[case["grad"]] * (n * k + n), "flops": 4 * rows * n * k}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_kept(x):
    """The values that an 8-bit checkpoint of x stands for, block by block of 64 columns."""
    got = []
    for piece in x.split(BLOCK, 1):
        most = piece.abs().max(1, keepdim=True).values
        step = most / 127
        got.append(torch.where(most < TINY, torch.zeros_like(piece), torch.round(piece / step) * step))
    return torch.cat(got, 1)


def _exact_phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def _exact_act(name, z):
    """(activation, derivative) of z."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        p = _exact_phi(z)
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    u = c * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(2 * u)  # (1 + tanh u) / 2
    return z * p, p + z * 2 * p * (1 - p) * c * (1 + 0.134145 * z.square())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    if op in ("ln_bwd", "lin_bwd") and case["ckpt"]:
        d["x"] = torch.cat([c * d["scales"][:, i: i + 1] for i, c in enumerate(d["codes"].split(BLOCK, 1))], 1)
    x = d["x"]
    if op == "ck":
        return _exact_act(case["act"], _exact_kept(x))[0]
    if op == "ln_fwd":
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(d["beta"], (x - mean[:, None]) * rstd[:, None], d["gamma"])
        return [y, mean, rstd] + ([_exact_kept(x)] if case["ckpt"] else [])
    if op == "ln_bwd":
        xh = (x - d["mean"].unsqueeze(1)) * d["rstd"].unsqueeze(1)
        g = d["dy"] * d["gamma"]
        proj = g.sum(1) / x.shape[1], (g * xh).sum(1) / x.shape[1]
        dx = (g - proj[0].unsqueeze(1) - xh * proj[1].unsqueeze(1)) * d["rstd"].unsqueeze(1)
        if case["add"]:
            dx += d["add"]
        return dx, torch.einsum("rc,rc->c", d["dy"], xh), torch.einsum("rc->c", d["dy"])
    if op == "lin_fwd":
        z = torch.addmm(d["bias"], x, d["w"].mT)
        y = _exact_act(case["act"], z)[0]
        if case["residual"]:
            y = y + d["residual"]
        return [y, _exact_kept(z)] if case["ckpt"] else [y]
    h, slope = _exact_act(case["act"], x)
    dx = torch.mm(d["dy"], d["w"]) * slope
    if case["add"]:
        dx += d["add"]
    return dx, torch.mm(d["dy"].mT, h), torch.mv(d["dy"].mT, torch.ones_like(d["dy"][:, 0]))
