"""The operators around the delta rule in 64 bits on the CPU, token by token, each
with a running bound of what 32-bit arithmetic may add.

U = 2^-24 is half a step of fp32.  A bound adds, for each fp32 result, a few U of
its size: GATE counts the roundings from the raw gate to a = exp(lambda) (sum,
exponential, logarithm or reciprocal, product: below 16, and the exponential turns
lambda's own error of a few U |lambda| into a relative one, 8 |lambda|), the
recurrences' other roundings (product, sum, and the same again where a tile is
folded and run a second time) are below 16 a token.  Whatever the order in which
runs of tokens are composed, each token's term goes through those.
Storage rounding is added last: half a step of the type, relative to the value."""

import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float32: U, torch.float64: 0.0}


def check(name, got, ref, err, kind=None):
    """|got - ref| <= err + half a storage step of ref, element by element."""
    got_ = got.detach().cpu().double()
    assert got_.shape == ref.shape, (name, got_.shape, ref.shape)
    assert torch.isfinite(got_).all(), f"{name}: not finite (unwritten?)"
    half = HALF[got.dtype if kind is None else kind]
    # the stored value is the rounding of a value within err of ref; smallest normals: 2^-126
    tol = err + half * (ref.abs() + err) + 2.0 ** -126
    off = (got_ - ref).abs()
    worst = float((off / tol).max()) if off.numel() else 0.0
    print(f"  {name}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3f} times the bound"


def gate(kind, g, A_log, dt_bias, gate_scale):
    """lambda, its derivatives by the raw gate and by A_log, and the relative error
    bound of a = exp(lambda); all broadcastable to [.., H, D]."""
    g = g.double()
    if kind == 0:
        lam = g.unsqueeze(-1)
        return lam, torch.ones_like(lam), torch.zeros_like(lam), (16 + 8 * lam.abs().clamp(max=1e4)) * U
    A, z = A_log.double().exp()[:, None], g + dt_bias.double()
    if kind == 1:
        lam = -A * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
        dz, dA = -A * torch.sigmoid(z), lam
    else:
        w = A * z
        p, pm = torch.sigmoid(w), torch.sigmoid(-w)
        lam, dz, dA = gate_scale * p, gate_scale * p * pm * A, gate_scale * p * pm * w
        # the sum z and the factor A each carry U, and the sigmoid's slope turns U |w| into lambda's error
    return lam, dz, dA, (16 + 8 * lam.abs() * (1 + A * z.abs())) * U


def scan(kind, x, g, A_log, dt_bias, h0, lengths, gate_scale=0.0, convex=False, dy=None, dht=None):
    """x [tokens, H, D] etc. on the CPU; returns {name: (value, error bound)}."""
    x = x.double()
    tokens, H, D = x.shape
    N = len(lengths)
    lam, sz, sA, rel = gate(kind, g, A_log, dt_bias, gate_scale)
    a = lam.exp().expand_as(x)
    rel = rel.expand_as(x)
    m = (-torch.expm1(lam)).expand_as(x) if convex else torch.ones_like(x)
    # 1 - exp: relative error a / (1 - a) times lambda's is below rel / m; series or difference add 8 U
    m_err = (a * rel + 8 * U * m.abs()) if convex else torch.zeros_like(x)
    zero = torch.zeros(N, H, D, dtype=torch.float64)
    h = zero.clone() if h0 is None else h0.double().clone()
    y, y_err, before, before_err = (torch.zeros_like(x) for _ in range(4))
    ht, ht_err = h.clone(), zero.clone()
    at = 0
    for n, L in enumerate(lengths):
        s, big, e = h[n], h[n].abs(), zero[n].clone()
        for t in range(at, at + L):
            before[t], before_err[t] = s, e
            u = m[t] * x[t]
            e = a[t] * e + (rel[t] + 16 * U) * a[t] * big + m_err[t] * x[t].abs() + 16 * U * u.abs()
            s, big = a[t] * s + u, a[t] * big + u.abs()
            y[t], y_err[t] = s, e
        ht[n], ht_err[n] = s, e
        at += L
    out = {"y": (y, y_err), "ht": (ht, ht_err)}
    if dy is None:
        return out
    dy = dy.double()
    r = zero.clone() if dht is None else dht.double().clone()
    ds, ds_err, ds_big = (torch.zeros_like(x) for _ in range(3))
    dh0, dh0_err = r.clone(), zero.clone()
    at = tokens
    for n in range(N - 1, -1, -1):
        c, big, e = r[n], r[n].abs(), zero[n].clone()
        for t in range(at - 1, at - 1 - lengths[n], -1):
            c, big = c + dy[t], big + dy[t].abs()
            e = e + 16 * U * big
            ds[t], ds_err[t], ds_big[t] = c, e, big
            e = a[t] * e + (rel[t] + 16 * U) * a[t] * big
            c, big = a[t] * c, a[t] * big
        dh0[n], dh0_err[n] = c, e
        at -= lengths[n]
    diff = before - x if convex else before
    size = before.abs() + x.abs() if convex else before.abs()
    dl = a * ds * diff
    dl_err = a * (ds_err * size + ds_big * (before_err + (rel + 16 * U) * size))
    dx = m * ds
    dx_err = m.abs() * ds_err + m_err * ds_big + 8 * U * ds_big * m.abs()
    out.update(dx=(dx, dx_err), dh0=(dh0, dh0_err))
    if kind == 0:
        out["dg"] = (dl.sum(-1), dl_err.sum(-1) + D * U * dl.abs().sum(-1))
        return out
    sz, sA = sz.expand_as(x), sA.expand_as(x)
    # the gate's slopes carry lambda's roundings too: below rel + 32 U relative
    dz, dz_err = dl * sz, dl_err * sz.abs() + (rel + 32 * U) * (dl * sz).abs()
    dA, dA_err = dl * sA, dl_err * sA.abs() + (rel + 32 * U) * (dl * sA).abs()
    out["dg"] = (dz, dz_err)
    # sums of at most 128 terms in fp32, the rest in 64 bits
    out["ddt_bias"] = (dz.sum(0), dz_err.sum(0) + 128 * U * dz.abs().sum(0))
    out["dA_log"] = (dA.sum((0, 2)), dA_err.sum((0, 2)) + 128 * U * dA.abs().sum((0, 2)))
    return out


def step_delta(kind, q, k, v, g, b, A_log, dt_bias, state, slots, scale, gate_scale=0.0):
    """Rows in order on a pool [P, H, D, D]; returns o, its error bound, which rows
    were written, the pool and its error bound."""
    N, H, D = v.shape
    G = H // k.shape[1]
    q, k, v = (t.double() for t in (q, k, v))
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    q = q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    k = k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    lam, _, _, rel = gate(kind, g, A_log, dt_bias, gate_scale)
    beta = torch.sigmoid(b.double())
    S, err = state.double().clone(), torch.zeros_like(state, dtype=torch.float64)
    o, o_err, wrote = torch.zeros_like(v), torch.zeros_like(v), torch.zeros(N, dtype=torch.bool)
    # norms of q and k: below D / 8 + 16 U relative each; a product over a row: D / 8 + 16 roundings
    d_ = (D / 8 + 32) * U
    for n in range(N):
        p = int(slots[n])
        if not 0 <= p < S.shape[0]:
            continue
        a = lam[n].exp().expand(H, D)[:, None, :]
        r = rel[n].expand(H, D)[:, None, :]
        e = a * err[p] + (r + U) * (a * S[p]).abs()
        M, kn, qn = a * S[p], k[n][:, None, :], q[n][:, None, :]
        got = (M * kn).sum(-1)
        got_err = (e * kn.abs()).sum(-1) + 2 * d_ * (M * kn).abs().sum(-1)
        d = beta[n][:, None] * (v[n] - got)
        dd = beta[n][:, None] * got_err + 16 * U * beta[n][:, None] * (v[n].abs() + got.abs())
        S[p] = M + d[..., None] * kn
        err[p] = e + dd[..., None] * kn.abs() + 2 * d_ * (d[..., None] * kn).abs() + 2 * U * M.abs()
        o[n] = scale * (S[p] * qn).sum(-1)
        # o is formed as S' q + d (k . q)
        size = (M * qn).abs().sum(-1) + d.abs() * (kn * qn).abs().sum(-1)
        o_err[n] = scale * ((err[p] * qn.abs()).sum(-1) + dd * (kn * qn).abs().sum(-1) + 4 * d_ * size)
        wrote[n] = True
    return o, o_err, wrote, S, err


def norm(x, res, w, eps, round_res=None):
    """r, y and the relative error bound of y: the sum of squares of a row held by up
    to 1024 threads with 32 values each takes 32 + 10 + 16 roundings, halved by the
    root; the other factors below 8."""
    r = x.double() if res is None else x.double() + res.double()
    rstd = 1 / (r.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    y = r * rstd * (1.0 if w is None else w.double())
    return r, rstd, y, 48 * U


def norm_bwd(r, w, dy, dres, eps):
    r, dy = r.double(), dy.double()
    w_ = torch.ones(r.shape[-1], dtype=torch.float64) if w is None else w.double()
    rstd = 1 / (r.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n = r * rstd
    dx = rstd * (w_ * dy - n * (n * w_ * dy).mean(-1, keepdim=True))
    size = rstd * ((w_ * dy).abs() + n.abs() * (n * w_ * dy).abs().mean(-1, keepdim=True))
    if dres is not None:
        dx, size = dx + dres.double(), size + dres.double().abs()
    rows = r.shape[0]
    dw = (dy * n).sum(0)
    # a thread adds its rows one by one, at most all of them
    dw_err = (64 + min(rows, 4096)) * U * (dy * n).abs().sum(0)
    return dx, 128 * U * size, dw, dw_err


def e4m3_ref(y, group):
    """scales and y / scale, in 64 bits."""
    rows, width = y.shape
    parts = y.split(group or width, -1)
    scales = torch.stack([(c.abs().amax(-1) / 448).clamp(min=2.0 ** -126) for c in parts], -1)
    z = torch.cat([c / scales[:, i:i + 1] for i, c in enumerate(parts)], -1)
    return scales, z


def lengths_of(total, cuts):
    c = [0] + sorted(cuts) + [total]
    return [b - a for a, b in zip(c, c[1:])]


def rand(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, dtype=torch.float64) * std


def gate_inputs(gen, kind, tokens, H, D, dt):
    if kind == 0:
        return (-0.1 * torch.nn.functional.softplus(rand(gen, tokens, H))).to(dt), None, None
    return (rand(gen, tokens, H, D).to(dt), (1.5 * torch.rand(H, generator=gen, dtype=torch.float64)).float(),
            rand(gen, H, D, std=0.5).float())
