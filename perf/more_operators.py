"""Linear attention with a decay for each head, and the 8-bit projections around it, as they are measured.

* ``lin``: S_t = exp(lambda_h) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t over packed or batched sequences, with grouped
  heads, forward and backward, and its single-token step on a pool of states;
* ``gemm``: the product of e4m3 matrices with a scale for each 128 of the contraction (activations: per row; weights: per
  block of 128 x 128), and a linear layer's training step on it;
* ``quant``: a matrix, or its transpose, as e4m3 with such scales.

``own`` chooses between the library's entry points and plain torch forms of the same operators.
"""

import math

import numpy as np
import torch

own = False

CHUNK = 64          # tokens per chunk of the plain linear attention
DEV = "cuda"
F8 = torch.float8_e4m3fn


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------

def _lin(name, op, B, T, H, Hk, D, dtype, seqs=0):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "Hk": Hk, "D": D, "dtype": dtype, "seqs": seqs}


def _step(name, N, H, Hk, D, dtype, pad):
    return {"name": name, "op": "lin_step", "N": N, "H": H, "Hk": Hk, "D": D, "dtype": dtype, "pad": pad}


def _gemm(name, op, M, N, K, dtype, block):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "dtype": dtype, "block": block}


def _quant(name, rows, cols, dtype, block, transpose):
    return {"name": name, "op": "quant", "rows": rows, "cols": cols, "dtype": dtype, "block": block,
            "transpose": transpose}


def listed():
    return [
        # training step of one layer on one long sequence, the headline size
        _lin("lin_train_t32768_h16_d128", "lin_train", 1, 32768, 16, 16, 128, "bf16"),
        # training on a pack of twelve uneven documents, 32 value heads on 8 key heads
        _lin("lin_train_varlen12_h32_gqa4", "lin_train", 1, 32768, 32, 8, 128, "bf16", seqs=12),
        # a small fp32 training problem with an odd length: a unit test's or a probe's size
        _lin("lin_train_f32_b2_t129_h2_d64", "lin_train", 2, 129, 2, 2, 64, "f32"),
        # prefill of a batch of prompts at an odd length
        _lin("lin_fwd_b4_t4095_h32_d128", "lin_fwd", 4, 4095, 32, 32, 128, "bf16"),
        # decoding one request: latency
        _step("lin_step_n1_h16_d128", 1, 16, 16, 128, "bf16", 0),
        # decoding a full serving batch with grouped heads and padding rows
        _step("lin_step_n250_gqa4_h32_d128", 250, 32, 8, 128, "bf16", 6),
        # a projection in decoding: one row
        _gemm("gemm_m1_n4096_k2048", "gemm", 1, 4096, 2048, "bf16", 128),
        # the same for a serving batch
        _gemm("gemm_m64_n4096_k4096", "gemm", 64, 4096, 4096, "bf16", 128),
        # prefill: 32768 tokens through a projection
        _gemm("gemm_m32768_n4096_k4096", "gemm", 32768, 4096, 4096, "bf16", 128),
        # no size a multiple of the tiles or of 16, fp32 output
        _gemm("gemm_f32_m1000_n2050_k4100", "gemm", 1000, 2050, 4100, "f32", 128),
        # training: a projection's forward and both gradients, activations quantised on the way
        _gemm("gemm_train_m8192_n4096_k2048", "gemm_train", 8192, 4096, 2048, "bf16", 128),
        # after an optimizer step: a weight for the backward's product
        _quant("quant_blocks_4096x4096_t", 4096, 4096, "bf16", 128, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["lin_train", "lin_fwd", "lin_step", "gemm", "gemm", "gemm_train", "quant"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("lin"):
        D, H = rng.choice([64, 128]), _log_int(rng, 1, 32)
        Hk = rng.choice([H, rng.choice([d for d in range(1, H + 1) if H % d == 0])])
        if op == "lin_step":
            N = _log_int(rng, 1, 250)
            return {"op": op, "N": N, "H": H, "Hk": Hk, "D": D, "dtype": dtype,
                    "pad": rng.choice([0, rng.randint(0, N - 1)])}
        tokens = _log_int(rng, 1, min(32768, (32768 if dtype == "bf16" else 16384) * 2048 // (H * D)))
        seqs = rng.choice([0, 0, rng.randint(1, min(tokens, 40))])
        B = 1 if seqs else min(tokens, rng.choice([1, 1, 2, 3, 4, 7]))
        return {"op": op, "B": B, "T": tokens // B, "H": H, "Hk": Hk, "D": D, "dtype": dtype, "seqs": seqs}

    def width():
        return rng.choice([128, 512, 1024, 2048, 4096, 16 * _log_int(rng, 1, 256), _log_int(rng, 1, 4096)])

    if op == "quant":
        cols = width()
        return {"op": op, "rows": _log_int(rng, 1, 32768 * 2048 // cols), "cols": cols, "dtype": dtype,
                "block": rng.choice([1, 128]), "transpose": rng.random() < 0.5}
    return {"op": op, "M": _log_int(rng, 1, 32768 if op == "gemm" else 8192), "N": width(), "K": width(),
            "dtype": dtype, "block": rng.choice([1, 128]) if op == "gemm" else 128}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """Lengths of the case's sequences: B equal ones, or `seqs` uneven ones (empty ones among them from eight on)."""
    if not case["seqs"]:
        return [case["T"]] * case["B"]
    n, total = case["seqs"], case["T"]
    r = np.random.RandomState(n * 7919 + total)
    cuts = np.sort(r.randint(0, total + 1, n - 1)) if n > 1 else np.zeros(0, np.int64)
    if n >= 8:
        cuts[1] = cuts[0]
    return [int(x) for x in np.diff(np.concatenate([[0], cuts, [total]]))]


# --------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------

def _rnd(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rnd(*shape):
        return torch.randn(shape, device=DEV, generator=gen)

    rnd.gen = gen
    return rnd


def _unit(x):
    """Rows of length one, as q and k are where a layer normalises them."""
    return x / x.norm(dim=-1, keepdim=True)


def _decay(rnd, H):
    """Log decays from fast to slow heads, -2^-1 to -2^-10 or so, none the same."""
    return -torch.exp2(-1.0 - 8.0 * torch.arange(H, device=DEV) / max(H - 1, 1) - torch.rand(H, device=DEV, generator=rnd.gen))


def _chunks(s, lens):
    """The plain form's plan: each sequence in chunks, with the token of each place."""
    rows, seq, at = [], [], 0
    for n, L in enumerate(lens):
        for a in range(0, L, CHUNK):
            rows.append((at + a, min(CHUNK, L - a), n))
        at += L
    start = torch.tensor([r[0] for r in rows], device=DEV, dtype=torch.int64)
    count = torch.tensor([r[1] for r in rows], device=DEV, dtype=torch.int64)
    place = torch.arange(CHUNK, device=DEV)
    s["on"] = place[None, :] < count[:, None]
    s["token"] = torch.where(s["on"], start[:, None] + place[None, :], start[:, None])
    s["start"], s["end"] = start, start + count
    s["seq"] = torch.tensor([r[2] for r in rows], device=DEV, dtype=torch.int64)
    s["bounds"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device=DEV, dtype=torch.int64)


def prepare(case, seed):
    rnd, dt, s, op = _rnd(seed), _dtype(case), {"case": case}, case["op"]
    if own:
        from chunked_gated_delta_bwd_amd import binding as G
        code = G.GDR_BF16 if case["dtype"] == "bf16" else G.GDR_F32
    if op in ("lin_train", "lin_fwd"):
        H, Hk, D, lens = case["H"], case["Hk"], case["D"], _lengths(case)
        T, N = sum(lens), len(lens)
        s["t"] = {"q": _unit(rnd(T, Hk, D)).to(dt), "k": _unit(rnd(T, Hk, D)).to(dt), "v": rnd(T, H, D).to(dt),
                  "log_decay": _decay(rnd, H), "h0": 0.1 * rnd(N, H, D, D)}
        if op == "lin_train":
            s["dO"], s["dht"] = rnd(T, H, D).to(dt), 0.1 * rnd(N, H, D, D)
        if own:
            cu = np.concatenate([[0], np.cumsum(lens)]).tolist() if case["seqs"] else None
            s["prob"] = G.LinProblem(case["B"], case["T"], H, D, N, code, scale=D ** -0.5, cu_seqlens=cu, Hk=Hk)
            s["ws"] = G.alloc_lin_workspace(s["prob"], DEV, backward=op == "lin_train")
            s["o"], s["ht"] = torch.empty_like(s["t"]["v"]), torch.empty_like(s["t"]["h0"])
            if op == "lin_train":
                s["out"] = {"d" + x: torch.empty_like(s["t"][x]) for x in ("q", "k", "v", "h0")}
        else:
            _chunks(s, lens)
    elif op == "lin_step":
        N, H, Hk, D, pad = case["N"], case["H"], case["Hk"], case["D"], case["pad"]
        s["t"] = {"q": _unit(rnd(N, Hk, D)).to(dt), "k": _unit(rnd(N, Hk, D)).to(dt), "v": rnd(N, H, D).to(dt),
                  "log_decay": _decay(rnd, H), "h0": None}
        # a pool of states a little larger than the batch, the rows' slots in no order, the last rows without one
        s["state"] = 0.3 * rnd(N + 3, H, D, D)
        s["slots"] = torch.randperm(N + 3, device=DEV, generator=rnd.gen)[:N].to(torch.int32)
        s["slots"][N - pad:] = -1
        s["rows"] = torch.arange(N - pad, device=DEV)
        s["o"] = torch.zeros(N, H, D, dtype=dt, device=DEV)
        if own:
            s["prob"] = G.LinProblem(N, 1, H, D, N, code, scale=D ** -0.5, Hk=Hk)
    elif op == "quant":
        rows, cols = case["rows"], case["cols"]
        s["x"] = (rnd(rows, cols) * torch.exp(rnd(rows, 1))).to(dt)
        if own:
            s["prob"] = G.QuantProblem(rows, cols, code, block=case["block"], transpose=case["transpose"])
            s["q"], s["scales"] = _quant_out(s["prob"])
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sa"] = _plain_quant(rnd(M, K) * torch.exp(0.5 * rnd(M, 1)), 1)
        s["b"], s["sb"] = _plain_quant(K ** -0.5 * rnd(N, K), case["block"])
        if own:
            s["prob"] = G.GemmProblem(M, N, K, code, block=case["block"])
            s["ws"] = G.alloc_gemm_workspace(s["prob"], DEV)
            s["c"] = torch.empty(M, N, dtype=dt, device=DEV)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        # activations and their gradient as the layer has them; the weight is quantised once for each product
        s["x"], s["dy"] = rnd(M, K).to(dt), (0.1 * rnd(M, N)).to(dt)
        w = K ** -0.5 * rnd(N, K)
        s["w"], s["sw"] = _plain_quant(w, 128)
        s["wt"], s["swt"] = _plain_quant(w.t().contiguous(), 128)
        if own:
            for x, shape in (("x", (M, K)), ("dy", (M, N))):
                for t in (False, True):
                    p = G.QuantProblem(*shape, code, block=1, transpose=t)
                    s[f"q{x}{int(t)}"] = (p, *_quant_out(p))
            for name, (m, n, k), block in (("y", (M, N, K), 128), ("dx", (M, K, N), 128), ("dw", (N, K, M), 1)):
                p = G.GemmProblem(m, n, k, G.GDR_F32 if name == "dw" else code, block=block)
                s["g" + name] = (p, G.alloc_gemm_workspace(p, DEV),
                                 torch.empty(m, n, dtype=torch.float32 if name == "dw" else dt, device=DEV))
    return s


def _quant_out(p):
    return torch.empty(p.q_shape, dtype=F8, device=DEV), torch.empty(p.scales_shape, device=DEV)


# --------------------------------------------------------------------------------------------------------------
# the operators
# --------------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op in ("lin_train", "lin_fwd"):
        return _plain_lin(s, op == "lin_train")
    if op == "lin_step":
        return _plain_step(s)
    if op == "quant":
        q, scales = _plain_quant(s["x"].float().t().contiguous() if s["case"]["transpose"] else s["x"], s["case"]["block"])
        return {"q": q, "scales": scales}
    if op == "gemm":
        return {"c": _plain_product(s["a"], s["sa"], s["b"], s["sb"], s["case"]["block"]).to(_dtype(s["case"]))}
    return _plain_train(s)


def _run_own(s, op):
    from chunked_gated_delta_bwd_amd import binding as G
    if op in ("lin_train", "lin_fwd"):
        G.gdr_lin_fwd(s["prob"], s["t"], s["ws"], s["o"], ht=s["ht"])
        if op == "lin_fwd":
            return {"o": s["o"], "ht": s["ht"]}
        G.gdr_lin_bwd(s["prob"], s["t"], s["dO"], s["dht"], s["ws"], s["out"])
        return {"o": s["o"], "ht": s["ht"], **s["out"]}
    if op == "lin_step":
        G.gdr_lin_step(s["prob"], s["t"], s["state"], s["o"], slots=s["slots"])
        return {"o": s["o"], "state": s["state"]}
    if op == "quant":
        G.gdr_quant(s["prob"], s["x"], s["q"], s["scales"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "gemm":
        G.gdr_gemm(s["prob"], s["a"], s["sa"], s["b"], s["sb"], s["c"], s["ws"])
        return {"c": s["c"]}
    for x in ("x", "dy"):
        for t in (0, 1):
            p, q, scales = s[f"q{x}{t}"]
            G.gdr_quant(p, s[x], q, scales)
    operands = {"y": (*s["qx0"][1:], s["w"], s["sw"]), "dx": (*s["qdy0"][1:], s["wt"], s["swt"]),
                "dw": (*s["qdy1"][1:], *s["qx1"][1:])}
    for name, (a, sa, b, sb) in operands.items():
        p, ws, c = s["g" + name]
        G.gdr_gemm(p, a, sa, b, sb, c, ws)
    return {name: s["g" + name][2] for name in operands}


def _between(lam, first, last, ok):
    """exp(lambda (last - first)) [H, ...] where ok, else 0; the exponent in 64 bits."""
    n = (last - first).double()
    return torch.where(ok, torch.exp(lam.double().view(-1, *[1] * n.dim()) * torch.where(ok, n, 0.0)), 0.0).float()


def _plain_lin(s, train):
    case, t = s["case"], s["t"]
    H, Hk, D, dt, scale = case["H"], case["Hk"], case["D"], _dtype(case), case["D"] ** -0.5
    lam, h0, on, start, end, seq, bounds = t["log_decay"], t["h0"], s["on"], s["start"], s["end"], s["seq"], s["bounds"]

    def split(x):                                     # [tokens, H or Hk, D] -> [H, chunks, CHUNK, D], zero past the end
        x = (x.float()[s["token"]] * on[:, :, None, None]).permute(2, 0, 1, 3)
        return x if x.shape[0] == H else x.repeat_interleave(H // Hk, 0)

    def join(x, heads):                               # back, summed over the heads that share one
        x = x.permute(1, 2, 0, 3)[on]
        return (x if heads == H else x.view(-1, heads, H // heads, D).sum(2)).to(dt)

    q, k, v = split(t["q"]), split(t["k"]), split(t["v"])
    pos = torch.arange(CHUNK, device=DEV)
    near = _between(lam, pos[None, :], pos[:, None], pos[:, None] >= pos[None, :])[:, None]     # [H, 1, i, j]
    # decay from each place to its chunk's last token, and from the token before the chunk to each place
    count = (end - start)[:, None]
    to_end = _between(lam, pos[None, :] + 1, count, pos[None, :] < count)[..., None]
    from_start = _between(lam, torch.zeros_like(pos), pos + 1, pos >= 0)[:, None, :, None]
    local = (v * to_end).transpose(-1, -2) @ k                                                   # [H, chunks, Dv, Dk]
    same = seq[:, None] == seq[None, :]
    chunk = torch.arange(len(seq), device=DEV)
    carry = _between(lam, end[None, :], start[:, None], same & (chunk[:, None] > chunk[None, :]))
    first = _between(lam, bounds[:-1][seq], start, seq >= 0)
    state = (carry @ local.flatten(2)).view_as(local) + first[..., None, None] * h0.transpose(0, 1)[:, seq]
    o = scale * (((q @ k.transpose(-1, -2)) * near) @ v + from_start * (q @ state.transpose(-1, -2)))
    member = seq[None, :] == torch.arange(len(h0), device=DEV)[:, None]
    whole = _between(lam, bounds[:-1], bounds[1:], bounds[1:] >= 0).t()[..., None, None]
    last = _between(lam, end[None, :], bounds[1:, None], member)
    ht = whole * h0 + (last @ local.flatten(2)).view(H, -1, D, D).transpose(0, 1)
    out = {"o": join(o, H), "ht": ht}
    if not train:
        return out
    dO = split(s["dO"])
    dlocal = scale * (dO * from_start).transpose(-1, -2) @ q
    dcarry = _between(lam, end[:, None], start[None, :], same & (chunk[:, None] < chunk[None, :]))
    dlast = _between(lam, end, bounds[1:][seq], seq >= 0)
    dstate = (dcarry @ dlocal.flatten(2)).view_as(local) + dlast[..., None, None] * s["dht"].transpose(0, 1)[:, seq]
    # decay from each place to the chunk's last token, that token's own place included
    qk, gv = (q @ k.transpose(-1, -2)) * near, (dO @ v.transpose(-1, -2)) * near
    dq = scale * (gv @ k + from_start * (dO @ state))
    dk = scale * (gv.transpose(-1, -2) @ q) + to_end * (v @ dstate)
    dv = scale * (qk.transpose(-1, -2) @ dO) + to_end * (k @ dstate.transpose(-1, -2))
    dfirst = _between(lam, bounds[:-1, None], start[None, :], member)
    dh0 = whole * s["dht"] + (dfirst @ dlocal.flatten(2)).view(H, -1, D, D).transpose(0, 1)
    return {**out, "dq": join(dq, Hk), "dk": join(dk, Hk), "dv": join(dv, H), "dh0": dh0}


def _plain_step(s):
    case, t, rows = s["case"], s["t"], s["rows"]
    G = case["H"] // case["Hk"]
    q, k = (t[x].float()[rows].repeat_interleave(G, 1) for x in ("q", "k"))
    slots = s["slots"][rows].long()
    st = s["state"][slots] * t["log_decay"].exp()[:, None, None] + t["v"].float()[rows][..., None] * k[:, :, None, :]
    s["state"][slots] = st
    s["o"][rows] = (case["D"] ** -0.5 * (st * q[:, :, None, :]).sum(-1)).to(s["o"].dtype)
    return {"o": s["o"], "state": s["state"]}


def _plain_quant(x, block):
    """e4m3 and the scales: for each row (block 1) or 128 rows (block 128) and 128 columns."""
    rows, cols = x.shape
    R, C = -(-rows // block), -(-cols // 128)
    y = torch.nn.functional.pad(x.float(), (0, 128 * C - cols, 0, block * R - rows)).view(R, block, C, 128)
    most = y.abs().amax((1, 3))
    # by a tensor: a division by a number may be a product with its reciprocal, one step off, and ties are common here
    scales = (most / torch.full_like(most, 448.0)).clamp(min=2.0 ** -126)
    q = (y / scales[:, None, :, None]).clamp(-448.0, 448.0).view(block * R, 128 * C)[:rows, :cols]
    return q.to(F8), scales


def _plain_values(q, scales, block):
    return q.float() * scales.repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(block, 0)[:q.shape[0]]


def _plain_product(a, sa, b, sb, block):
    return _plain_values(a, sa, 1) @ _plain_values(b, sb, block).t()


def _plain_train(s):
    x, dy, dt = s["x"].float(), s["dy"].float(), _dtype(s["case"])
    return {"y": _plain_product(*_plain_quant(x, 1), s["w"], s["sw"], 128).to(dt),
            "dx": _plain_product(*_plain_quant(dy, 1), s["wt"], s["swt"], 128).to(dt),
            "dw": _plain_product(*_plain_quant(dy.t().contiguous(), 1), *_plain_quant(x.t().contiguous(), 1), 1)}


# --------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------------

def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op in ("lin_train", "lin_fwd"):
        H, Hk, D, N = case["H"], case["Hk"], case["D"], len(_lengths(case))
        T, st = sum(_lengths(case)), 4 * N * H * D * D
        # per token and head: the state's update and its product with the query
        if op == "lin_fwd":
            return {"bytes": e * T * D * (2 * Hk + 2 * H) + 2 * st + 4 * H, "flops": 4 * T * H * D * D}
        # backward: the states again, their gradient, and a product with each for dq, dk, dv
        return {"bytes": e * T * D * (4 * Hk + 4 * H) + 4 * st + 4 * H, "flops": 14 * T * H * D * D}
    if op == "lin_step":
        on, H, Hk, D = case["N"] - case["pad"], case["H"], case["Hk"], case["D"]
        return {"bytes": 8 * on * H * D * D + e * on * D * (2 * Hk + 2 * H) + 4 * case["N"] + 4 * H,
                "flops": 5 * on * H * D * D}
    if op == "quant":
        r, c = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        return {"bytes": r * c * (e + 1) + 4 * -(-r // case["block"]) * -(-c // 128), "flops": 2 * r * c}
    M, N, K = case["M"], case["N"], case["K"]
    G = -(-K // 128)
    if op == "gemm":
        return {"bytes": M * K + N * K + e * M * N + 4 * G * (M + -(-N // case["block"])), "flops": 2 * M * N * K}
    return {"bytes": e * 2 * M * (K + N) + 2 * N * K + 4 * N * K + 8 * G * -(-N // 128), "flops": 6 * M * N * K}


# --------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("lin_train", "lin_fwd"):
        return _exact_lin(case, s)
    if op == "lin_step":
        return _exact_step(case, s)
    if op == "quant":
        q, scales, _ = _exact_quant(s["x"].t() if case["transpose"] else s["x"], case["block"])
        return {"q": q, "scales": scales}
    if op == "gemm":
        return {"c": _exact_product(s["a"], s["sa"], 1, s["b"], s["sb"], case["block"])}
    a, b = {}, {}
    for n in ("x", "dy"):
        for t, m in ((0, s[n]), (1, s[n].t())):
            _, scales, q = _exact_quant(m, 1)
            a[n, t] = (q, scales, 1)
    b["w"], b["wt"] = (s["w"], s["sw"], 128), (s["wt"], s["swt"], 128)
    return {"y": _exact_product(*a["x", 0], *b["w"]), "dx": _exact_product(*a["dy", 0], *b["wt"]),
            "dw": _exact_product(*a["dy", 1], *a["x", 1])}


def _exact_lin(case, s):
    """Every pair of tokens, head by head: o_i = scale (sum_{j <= i} e^{(i - j) lambda} (q_i . k_j) v_j + e^{(i + 1) lambda} h0 q_i)."""
    t, train, scale, G = s["t"], case["op"] == "lin_train", case["D"] ** -0.5, case["H"] // case["Hk"]
    names = ["o", "ht"] + (["dq", "dk", "dv", "dh0"] if train else [])
    like = {"o": "v", "ht": "h0", "dq": "q", "dk": "k", "dv": "v", "dh0": "h0"}
    out = {n: torch.zeros(t[like[n]].shape, dtype=torch.float64, device=DEV) for n in names}
    at, most = 0, 4096
    for n, L in enumerate(_lengths(case)):
        here = slice(at, at + L)
        at += L
        i = torch.arange(L, device=DEV, dtype=torch.float64)
        for h in range(case["H"]):
            lam, S0 = t["log_decay"][h].double(), t["h0"][n, h].double()
            q, k, v = t["q"][here, h // G].double(), t["k"][here, h // G].double(), t["v"][here, h].double()
            rise, left = torch.exp(lam * (i + 1))[:, None], torch.exp(lam * (L - 1 - i))[:, None]
            out["ht"][n, h] = torch.exp(lam * L) * S0 + (left * v).t() @ k
            if train:
                R0, dO = s["dht"][n, h].double(), s["dO"][here, h].double()
                out["dh0"][n, h] = torch.exp(lam * L) * R0 + scale * (rise * dO).t() @ q
                out["dk"][here, h // G] += left * (v @ R0)
                out["dv"][here, h] += left * (k @ R0.t())
            for r in range(0, L, most):
                rows, upto = slice(r, min(L, r + most)), min(L, r + most)
                gap = i[rows, None] - i[None, :upto]
                w = scale * torch.where(gap >= 0, torch.exp(lam * gap.clamp(min=0)), 0.0)
                pair = w * (q[rows] @ k[:upto].t())
                out["o"][here, h][rows] = pair @ v[:upto] + scale * rise[rows] * (q[rows] @ S0.t())
                if train:
                    grad = w * (dO[rows] @ v[:upto].t())
                    out["dq"][here, h // G][rows] += grad @ k[:upto] + scale * rise[rows] * (dO[rows] @ S0)
                    out["dk"][here, h // G][:upto] += grad.t() @ q[rows]
                    out["dv"][here, h][:upto] += pair.t() @ dO[rows]
    return out


def _exact_step(case, s):
    t, on = s["t"], s["rows"].numel()
    head = torch.arange(case["H"], device=DEV) // (case["H"] // case["Hk"])
    q, k, v = t["q"].double()[:on, head], t["k"].double()[:on, head], t["v"].double()[:on]
    st, o, at = s["state"].double(), s["o"].double(), s["slots"][:on].long()
    st[at] = torch.exp(t["log_decay"].double())[:, None, None] * st[at] + torch.matmul(v.unsqueeze(-1), k.unsqueeze(-2))
    o[:on] = case["D"] ** -0.5 * torch.matmul(st[at], q.unsqueeze(-1)).squeeze(-1)
    return {"o": o, "state": st}


def _exact_quant(x, block):
    """x over its scales, the scales as they are stored (fp32), and the quotient as it is stored (to nearest even)."""
    x = x.double()
    scales = torch.stack([torch.stack([b.abs().amax(-1) if block == 1 else b.abs().amax().view(1) for b in r.split(128, 1)], -1)
                          for r in x.split(x.shape[0] if block == 1 else 128, 0)]).flatten(0, 1)
    scales = (scales / 448).clamp(min=2.0 ** -126).float()
    z = x.clone()
    for g in range(scales.shape[1]):
        z[:, 128 * g:128 * (g + 1)] /= scales[:, g].double().repeat_interleave(block)[:x.shape[0], None]
    return z, scales.double(), z.float().to(F8)


def _exact_product(a, sa, a_block, b, sb, b_block):
    c = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=DEV)
    most = 128 * max(1, 2 ** 28 // (128 * max(c.shape)))
    for g0 in range(0, a.shape[1], most):
        x, y = a[:, g0:g0 + most].double(), b[:, g0:g0 + most].double()
        for m, scales, block in ((x, sa, a_block), (y, sb, b_block)):
            for g in range(0, m.shape[1], 128):
                m[:, g:g + 128] *= scales[:, (g0 + g) // 128].double().repeat_interleave(block)[:m.shape[0], None]
        c += x @ y.t()
    return c
