"""Linear attention with a decay for each head, and the e4m3 product, in 64 bits on the
CPU, with a bound of what the library's arithmetic may add.

U = 2^-24 is half a step of fp32, HALF (layer_ref) half a step of a type.  Blocks are 64
tokens from each sequence's start.  With bf16 tensors the library rounds to bf16, by half
a step (2^-8) each, the pairs' products within a block and the state at a block's start
where it meets the query.  What it adds to a state is in two bf16 parts (2^-16 is left),
in three (24 bits, as fp32) where the state is returned.  Everything else is fp32: a
product over D channels or 64 tokens adds one U a term, decays are exponentials of
n lambda (the product rounds by U n |lambda|, the exponential by a few U), and a state that
passes nb blocks is decayed and added to nb times.  Each bound is taken of the sum of the
terms' magnitudes, since terms may cancel."""

import torch

import layer_ref as R

U = R.U
BLOCK = 64


def _factors(x, lam, nb):
    low = x.dtype is torch.bfloat16
    D = x.shape[-1]
    fp32 = (2 * D + 3 * BLOCK + 8 * nb + 32 + 16 * BLOCK * min(abs(float(lam)), 8.0)) * U
    return (2.0 ** -8 if low else 0.0), fp32


def role(x, y, z, init, lam, out_first, reverse=False):
    """One head of one sequence: out_i = sum_j c^|i-j| (x_i . y_j) z_j + c^m init x_i over the
    tokens j up to i (from i on, reversed), m = i + 1 tokens from the start (L - 1 - i to
    the end, reversed); and the state after the last token (before the first).  init:
    [channels of z, channels of y].  Values and error bounds; out_first: factor of the
    pairs, the state's additions and init's share as a triple."""
    pair_f, add_f, init_f = out_first
    L, lam = x.shape[0], float(lam)
    nb = -(-L // BLOCK) if L else 0
    h, f = _factors(x, lam, nb)
    xd, yd, zd = x.double(), y.double(), z.double()
    S0 = torch.zeros(z.shape[1], y.shape[1], dtype=torch.float64) if init is None else init.double()
    i = torch.arange(L, dtype=torch.float64)
    gap = i[None, :] - i[:, None] if reverse else i[:, None] - i[None, :]
    W = torch.where(gap >= 0, torch.exp(lam * gap.clamp(min=0)) if lam > -1e30 else (gap == 0).double(), 0.0)
    pw = lambda n: torch.exp(lam * n) if lam > -1e30 else (n == 0).double()  # noqa: E731
    near = (i[:, None] // BLOCK == i[None, :] // BLOCK).double()
    m = L - 1 - i if reverse else i + 1
    pair = pair_f * (xd @ yd.t()) * W
    size = abs(pair_f) * (xd.abs() @ yd.abs().t()) * W
    out = pair @ zd + init_f * pw(m)[:, None] * (xd @ S0.t())
    total = size @ zd.abs() + abs(init_f) * pw(m)[:, None] * (xd.abs() @ S0.abs().t())
    err = f * total + h * ((pair * near).abs() @ zd.abs())
    # the state that each block starts from, rounded where it meets x
    for b in range(nb):
        rows = (i // BLOCK == b)
        at = min(L, (b + 1) * BLOCK) - 1 if reverse else b * BLOCK
        before = (i > at) if reverse else (i < at)
        n = (i - at) if reverse else (at - 1 - i)
        w = torch.where(before, pw(n.clamp(min=0)), 0.0)
        S = add_f * (w[:, None] * zd).t() @ yd + pw(torch.tensor(float(L - 1 - at if reverse else at), dtype=torch.float64)) * S0
        A = abs(add_f) * (w[:, None] * zd.abs()).t() @ yd.abs()     # what was added, terms' sizes
        mm = (at - i if reverse else i - at + 1)[rows]
        err[rows] += h * abs(init_f) * pw(mm)[:, None] * (xd[rows].abs() @ (S.abs() + 2.0 ** -8 * A).t())
    left = i + 1 if reverse else L - 1 - i
    whole = pw(torch.tensor(float(L), dtype=torch.float64))
    end = add_f * (pw(left)[:, None] * zd).t() @ yd + whole * S0
    end_err = f * (abs(add_f) * (pw(left)[:, None] * zd.abs()).t() @ yd.abs() + whole * S0.abs())
    return out, err, end, end_err


def lin(q, k, v, log_decay, h0, lengths, scale, dO=None, dht=None):
    """q, k [T, Hk, D], v [T, H, D] etc. on the CPU; {name: (value, error bound)}."""
    T, H, D = v.shape
    Hk, N = q.shape[1], len(lengths)
    G = H // Hk
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    shapes = {"o": (T, H, D), "ht": (N, H, D, D), "dq": (T, Hk, D), "dk": (T, Hk, D), "dv": (T, H, D), "dh0": (N, H, D, D)}
    out = {n: (z(*s), z(*s)) for n, s in shapes.items() if dO is not None or n in ("o", "ht")}

    def put(name, at, value, err):
        out[name][0][at] += value
        # a sum over value heads: one rounding of the running sum each
        out[name][1][at] += err + (U * G * value.abs() if G > 1 else 0.0)

    at = 0
    for n, L in enumerate(lengths):
        s = slice(at, at + L)
        at += L
        for h in range(H):
            lam, a, b, c = log_decay[h], q[s, h // G], k[s, h // G], v[s, h]
            S0 = None if h0 is None else h0[n, h]
            o, e, end, end_e = role(a, b, c, S0, lam, (scale, 1.0, scale))
            put("o", (s, h), o, e)
            put("ht", (n, h), end, end_e)
            if dO is None:
                continue
            g, R0 = dO[s, h], None if dht is None else dht[n, h]
            t = lambda m: None if m is None else m.t()  # noqa: E731
            o, e, _, _ = role(g, c, b, t(S0), lam, (scale, 1.0, scale))
            put("dq", (s, h // G), o, e)
            o, e, _, _ = role(c, g, a, t(R0), lam, (scale, scale, 1.0), True)
            put("dk", (s, h // G), o, e)
            o, e, end, end_e = role(b, a, g, R0, lam, (scale, scale, 1.0), True)
            put("dv", (s, h), o, e)
            put("dh0", (n, h), end, end_e)
    return out


def tokens(q, k, v, log_decay, h0, lengths, scale):
    """The recurrence token by token, in 64 bits, as autograd can follow it: o, ht."""
    H, G = v.shape[1], v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    rows, ends, at = [], [], 0
    for n, L in enumerate(lengths):
        S = h0[n]
        for t in range(at, at + L):
            S = torch.exp(log_decay)[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            rows.append(scale * (S * q[t][:, None, :]).sum(-1))
        ends.append(S)
        at += L
    return torch.stack(rows) if rows else v, torch.stack(ends)


def product(a, sa, b, sb, block, dtype=torch.float32):
    """c and its error bound.  fp32 results: a group's 128 products are exact and their sum may
    round once a term, as may the sum over groups; two roundings of the scales' product.  bf16
    results take instructions that align the products of a few (at most 8) elements to the
    largest of them and drop what is 2^-13 below it: at most 8 x 2^-13 of that largest, so
    2^-10 of the sum of the magnitudes."""
    K = a.shape[1]
    x = a.float().double() * sa.double().repeat_interleave(128, 1)[:, :K]
    y = b.float().double() * sb.double().repeat_interleave(128, 1)[:, :K].repeat_interleave(block, 0)[:b.shape[0]]
    size = x.abs() @ y.abs().t()
    return x @ y.t(), ((128 + sa.shape[1] + 16) * U + (2.0 ** -10 if dtype is torch.bfloat16 else 0.0)) * size


def quantised(y, block):
    """Bytes and scales of y [R, C] (fp32 or bf16): quotients rounded to fp32 once, then to e4m3."""
    Rn, C = y.shape
    R_, C_ = -(-Rn // block), -(-C // 128)
    p = torch.nn.functional.pad(y.double(), (0, 128 * C_ - C, 0, block * R_ - Rn)).view(R_, block, C_, 128)
    scales = (p.abs().amax((1, 3)) / 448).float().clamp(min=2.0 ** -126)
    z = (p / scales.double()[:, None, :, None]).float().view(block * R_, 128 * C_)[:Rn, :C]
    return z.to(torch.float8_e4m3fn), scales
