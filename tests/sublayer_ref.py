"""The gated linear layer, dropout and the residual norm in 64 bits, with how far the operators may be off.

Tolerances are those of test_gpu_layers, with u the unit roundoff of a type:
* a product of K terms summed in fp32 is within K 2^-23 sum |a b|, an activation within 2^-20 (1 + |g|) with a slope of at most 1.13, a
  derivative within 2^-20 (1 + |g|);
* of a product of two values each passes its error on with the other's size, the two errors' own product is below 1% of that;
* a row's fp32 statistics and normalised values: depth 2^-22 (1 + max|v| rstd) (1 + |vhat|), with `depth` the additions one value
  goes through: at most 80, and one for every 256 columns;
* what reaches a norm with an error e is normalised with (2 + |vhat|) rstd max(e) more.
"""
import math

import torch

import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L

EPS = 1e-5


def act64(act, g):
    return g * torch.sigmoid(g) if act == L.ACT_SILU else base.act64(act, g)


def slope64(act, g):
    if act != L.ACT_SILU:
        return base.slope64(act, g)
    q = torch.sigmoid(g)
    return q + g * q * (1 - q)


def gated(x, w, b, act):
    """(h, g, u) and how far each may be off before its rounding."""
    n, k = w.shape[0] // 2, x.shape[1]
    x, w = x.double(), w.double()
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    e = (k + 2) * 2.0 ** -23 * size
    g, u, eg, eu = z[:, :n], z[:, n:], e[:, :n], e[:, n:]
    a = act64(act, g)
    eh = 1.01 * ((1.13 * eg + 2.0 ** -20 * (1 + g.abs())) * u.abs() + a.abs() * eu) + 2.0 ** -23 * (a * u).abs()
    return (a * u, eh), (g, eg), (u, eu)


def gated_grads(dy, g, u, w, act, dtype):
    """(dz, dw, db) and how far each may be off before its rounding; h is rounded to dtype."""
    out, rows = w.shape[0], dy.shape[0]
    dy, w = dy.double(), w.double()
    dh, ed = dy @ w, (out + 2) * 2.0 ** -23 * (dy.abs() @ w.abs())
    a, s, ea = act64(act, g), slope64(act, g), 2.0 ** -20 * (1 + g.abs())
    dg, du, h = dh * u * s, dh * a, a * u
    edg = 1.01 * (ed * (u * s).abs() + (dh * u).abs() * ea) + 2.0 ** -22 * dg.abs()
    edu = 1.01 * (ed * a.abs() + dh.abs() * ea) + 2.0 ** -22 * du.abs()
    eh = base.U[dtype] * 1.01 * h.abs() + ea * u.abs() + 2.0 ** -25
    ew = dy.abs().t() @ (eh + (rows + 2) * 2.0 ** -23 * h.abs())
    return (torch.cat([dg, du], 1), torch.cat([edg, edu], 1)), (dy.t() @ h, ew), (dy.sum(0), rows * 2.0 ** -23 * dy.abs().sum(0))


# ---------------------------------------------------------------- dropout


def philox(counter, key):
    """Philox4x32-10 on Python's whole numbers or tensors of int64: products of 32 by 16 bits stay exact."""
    def product(m, x):
        lo, hi = m * (x & 0xFFFF), m * (x >> 16)  # below 2^48 each
        t = (lo >> 16) + hi
        return t >> 16, ((t & 0xFFFF) << 16) | (lo & 0xFFFF)

    a, b, c, d = counter
    k0, k1 = key
    for i in range(10):
        (h0, l0), (h1, l1) = product(0xD2511F53, a), product(0xCD9E8D57, c)
        a, b, c, d = h1 ^ b ^ (k0 + i * 0x9E3779B9) % 2 ** 32, l1, h0 ^ d ^ (k1 + i * 0xBB67AE85) % 2 ** 32, l0
    return a, b, c, d


def stays(rows, cols, p, key, site, first_row=0):
    seed, step = (int(v) % 2 ** 64 for v in key.tolist())
    groups = -(-cols // 8)
    i = torch.arange(first_row * groups, (first_row + rows) * groups, device=key.device)
    words = philox((i % 2 ** 32, i // 2 ** 32, torch.full_like(i, step % 2 ** 32), torch.full_like(i, site)), (seed % 2 ** 32, seed // 2 ** 32))
    bits = torch.stack([part for w in words for part in (w % 65536, w // 65536)], 1)
    return bits.reshape(rows, groups * 8)[:, :cols] >= round(p * 65536)


def factor(p):
    return 65536 / (65536 - round(p * 65536))


# ---------------------------------------------------------------- the residual sum and its norms


def depth(cols):
    return 80 + cols // 256


def norm64(v, layer):
    """(vhat, mean, rstd) and vhat's error for an exact v."""
    mean = v.mean(1) if layer else torch.zeros_like(v[:, 0])
    c = v - mean[:, None]
    rstd = 1 / (c.square().mean(1) + EPS).sqrt()
    hat = c * rstd[:, None]
    return hat, mean, rstd, depth(v.shape[1]) * 2.0 ** -22 * (1 + v.abs().amax(1) * rstd)[:, None] * (1 + hat.abs())


def residual_norm(x, block, p, layer, through):
    """{name: (value, error before its rounding)}; p holds the parameters (or None), `through` is scale * factor or 0."""
    got, d = {}, {k: None if v is None else v.double() for k, v in p.items()}
    s, es = x.double(), torch.zeros_like(x, dtype=torch.float64)
    if block is not None:
        n = block.double()
        en = torch.zeros_like(n)
        if d["block_gamma"] is not None:
            hat, mean, rstd, eh = norm64(n, layer)
            got["block_mean"], got["block_rstd"] = (mean, 80 * 2.0 ** -24 * n.abs().amax(1)), (rstd, depth(n.shape[1]) * 2.0 ** -22 * rstd * (1 + n.abs().amax(1) * rstd))
            n, en = hat * d["block_gamma"], eh * d["block_gamma"].abs()
            if layer:
                n, en = n + d["block_beta"], en + 2.0 ** -22 * d["block_beta"].abs()
        c = through * (d["gate"] if d["gate"] is not None else 1.0)
        got["n"] = (n, en)
        s, es = s + c * n, c.abs() * en + 2.0 ** -22 * (s.abs() + (c * n).abs())
    got["s"] = (s, es)
    if d["gamma"] is not None:
        hat, mean, rstd, eh = norm64(s, layer)
        worst = es.amax(1)
        got["mean"] = (mean, depth(s.shape[1]) * 2.0 ** -24 * s.abs().amax(1) + worst)
        got["rstd"] = (rstd, rstd * (depth(s.shape[1]) * 2.0 ** -22 * (1 + s.abs().amax(1) * rstd) + rstd * worst))
        y, ey = hat * d["gamma"], (eh + (2 + hat.abs()) * (rstd * worst)[:, None]) * d["gamma"].abs()
        if layer:
            y, ey = y + d["beta"], ey + 2.0 ** -22 * d["beta"].abs()
        got["y"] = (y, ey)
    return got


def _norm_back(f, hat, rstd, layer, spread, ef):
    """A norm's backward pass from f, known to +-ef: (value, error)."""
    m = f.mean(1, keepdim=True) if layer else torch.zeros_like(f[:, :1])
    r = rstd[:, None]
    out = r * (f - m - hat * (f * hat).mean(1, keepdim=True))
    size = r * (f.abs() + f.abs().mean(1, keepdim=True) + hat.abs() * (f * hat).abs().mean(1, keepdim=True))
    passed = r * (ef + ef.mean(1, keepdim=True) + hat.abs() * (ef * hat.abs()).mean(1, keepdim=True))
    return out, depth(f.shape[1]) * 2.0 ** -21 * spread * size + passed


def residual_norm_grads(dy, ds, s, block, p, stats, layer, through):
    """{name: (value, error before its rounding)}; stats: the forward pass's mean, rstd, block_mean, block_rstd (or None)."""
    got, d = {}, {k: None if v is None else v.double() for k, v in p.items()}
    st = {k: None if v is None else v.double() for k, v in stats.items()}
    some = ds if dy is None else dy
    rows = some.shape[0]
    m = (min(rows, 512) + 32) * 2.0 ** -24

    def standard(v, mean, rstd):
        v = v.double()
        return (v - (mean[:, None] if layer else 0.0)) * rstd[:, None], 1 + (v.abs().amax(1) * rstd)[:, None]

    t = ds.double() if ds is not None else torch.zeros_like(some, dtype=torch.float64)
    et = torch.zeros_like(t)
    if d["gamma"] is not None:
        hat, spread = standard(s, st["mean"], st["rstd"])
        q = dy.double()
        back, eb = _norm_back(q * d["gamma"], hat, st["rstd"], layer, spread, 0 * q)
        t, et = t + back, eb + 2.0 ** -22 * t.abs()
        got["dgamma"] = (q * hat).sum(0), (m * (q * hat).abs() + 2.0 ** -21 * spread * q.abs()).sum(0)
        if layer:
            got["dbeta"] = q.sum(0), m * q.abs().sum(0)
    got["dx"] = t, et
    if through is None:
        return got
    e, ee = t * through, et * through.abs() + 2.0 ** -22 * (t * through).abs()
    gate = d["gate"] if d["gate"] is not None else 1.0
    f, ef = e * gate, ee * abs(gate) + 2.0 ** -22 * (e * gate).abs()
    n = en = None
    if d["block_gamma"] is not None:
        hat, spread = standard(block, st["block_mean"], st["block_rstd"])
        got["dblock_gamma"] = (f * hat).sum(0), (ef * hat.abs() + f.abs() * 2.0 ** -21 * spread + m * (f * hat).abs()).sum(0)
        if layer:
            got["dblock_beta"] = f.sum(0), (ef + m * f.abs()).sum(0)
        n, en = hat * d["block_gamma"], 2.0 ** -21 * spread * (hat * d["block_gamma"]).abs() + 2.0 ** -21 * spread * d["block_gamma"].abs()
        if layer:
            n, en = n + d["block_beta"], en + 2.0 ** -22 * d["block_beta"].abs()
        f, ef = f * d["block_gamma"], ef * d["block_gamma"].abs() + 2.0 ** -22 * (f * d["block_gamma"]).abs()
        got["dblock"] = _norm_back(f, hat, st["block_rstd"], layer, spread, ef)
    else:
        got["dblock"] = f, ef
        if block is not None:
            n, en = block.double(), 0.0
    if d["gate"] is not None:
        # from the sums of d bhat and d, each with its own error, so that the parts' sizes count and not only their sum's
        size = n.abs() if d["block_gamma"] is None else (hat * d["block_gamma"]).abs() + (d["block_beta"].abs() if layer else 0.0)
        got["dgate"] = (e * n).sum(0), (ee * size + e.abs() * en + 2 * m * e.abs() * size).sum(0)
    return got


def check(got, want, dtype, what):
    value, error = want
    base._within(got, value, base._rounding(value, dtype) + base.U[dtype] * error + error + 1e-38, what)
