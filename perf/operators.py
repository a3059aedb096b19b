"""The recurrent layer's operators beside the chunked delta rule, as they are measured.

Three operators of one layer, in training and in serving:

* ``scan``: the gated linear recurrence s_t = exp(lambda_t) s_{t-1} + u_t per channel, forward and backward over
  packed or batched sequences, and its single-token step on a pool of states;
* ``norm``: the root-mean-square norm with the residual's addition, its backward, and the form whose output is
  e4m3 with scales;
* ``step``: the gated delta rule's single-token step on a pool of states.

``own`` chooses between the library's entry points and plain torch forms of the same operators.
"""

import math

import numpy as np
import torch

own = False

SCALAR, CHANNEL, SIGMOID = 0, 1, 2     # gate kinds: log decay per head, softplus and bounded sigmoid per channel
GATE_SCALE = -2.0                      # bound of the sigmoid gate's log decay
EPS = 1e-6
DEV = "cuda"


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------

def _scan(name, op, B, T, H, D, gate, convex, dtype, seqs=0):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "D": D, "gate": gate, "convex": convex, "dtype": dtype,
            "seqs": seqs}


def _norm(name, op, rows, width, dtype, res, group=0):
    return {"name": name, "op": op, "rows": rows, "width": width, "dtype": dtype, "res": res, "group": group}


def _step(name, N, H, Hk, D, gate, dtype, pad):
    return {"name": name, "op": "step", "N": N, "H": H, "Hk": Hk, "D": D, "gate": gate, "dtype": dtype, "pad": pad}


def listed():
    return [
        # training step of one layer on one long sequence, the headline size: per-channel softplus gate
        _scan("scan_train_t32768_h16_d128", "scan_train", 1, 32768, 16, 128, CHANNEL, False, "bf16"),
        # training on a pack of twelve uneven documents with 32 heads, one decay per head, convex input
        _scan("scan_train_varlen12_h32_d128", "scan_train", 1, 32768, 32, 128, SCALAR, True, "bf16", seqs=12),
        # a small fp32 training problem with an odd length: a unit test's or a probe's size
        _scan("scan_train_f32_b2_t129_h2_d64", "scan_train", 2, 129, 2, 64, SIGMOID, False, "f32"),
        # prefill of a batch at an odd length with plain per-channel decays and no gate function (D = 1)
        _scan("scan_fwd_b2_t4095_c2050", "scan_fwd", 2, 4095, 2050, 1, SCALAR, False, "bf16"),
        # one decoding step of a serving batch: 64 requests, some rows padding
        _scan("scan_step_n64_h32_d128", "scan_step", 64, 1, 32, 128, CHANNEL, True, "bf16"),
        # training: the block's norm at model width with the residual's addition
        _norm("norm_train_8192x2048_res", "norm_train", 8192, 2048, "bf16", True),
        # training: the norm of every head's output row of the delta rule (32768 tokens, 16 heads of 128)
        _norm("norm_train_heads_524288x128", "norm_train", 524288, 128, "bf16", False),
        # prefill with an 8-bit projection behind the norm, a scale for each 128 channels
        _norm("norm_e4m3_32768x4096_res_g128", "norm_quant", 32768, 4096, "bf16", True, 128),
        # decoding: four rows, one scale a row
        _norm("norm_e4m3_4x2048_res", "norm_quant", 4, 2048, "bf16", True, 0),
        # decoding one request: latency
        _step("step_n1_h16_d128", 1, 16, 16, 128, SCALAR, "bf16", 0),
        # decoding a full serving batch with grouped heads and padding rows
        _step("step_n250_gqa4_h32_d128", 250, 32, 8, 128, SCALAR, "bf16", 6),
        # a per-channel gate with 64-wide heads in fp32
        _step("step_kda_n33_h16_d64_f32", 33, 16, 16, 64, CHANNEL, "f32", 1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["scan_train", "scan_fwd", "scan_step", "norm_train", "norm_quant", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("scan"):
        gate = rng.choice([SCALAR, CHANNEL, SIGMOID])
        D = rng.choice([1, 1, 8, 24, 40, 64, 96, 128, 128, 200, 256])
        H = _log_int(rng, 1, 4096 // D)
        if op == "scan_step":
            B, T, seqs = _log_int(rng, 1, 256), 1, 0
        else:
            tokens = _log_int(rng, 1, min(32768, (32768 if dtype == "bf16" else 16384) * 2048 // (H * D)))
            seqs = rng.choice([0, 0, rng.randint(1, min(tokens, 40))])
            B = 1 if seqs else min(tokens, rng.choice([1, 1, 2, 3, 4, 7]))
            T = tokens // B
        return {"op": op, "B": B, "T": T, "H": H, "D": D, "gate": gate, "convex": rng.random() < 0.5, "dtype": dtype,
                "seqs": seqs}
    if op.startswith("norm"):
        width = rng.choice([64, 128, 1024, 2048, 4096, _log_int(rng, 1, 8192)])
        most = 32768 * (4096 if op == "norm_quant" else 2048) // (1 if dtype == "bf16" else 2)
        rows = _log_int(rng, 1, most // width)
        return {"op": op, "rows": rows, "width": width, "dtype": dtype, "res": rng.random() < 0.7,
                "group": rng.choice([0, 128]) if op == "norm_quant" else 0}
    H = _log_int(rng, 1, 32)
    divs = [d for d in range(1, H + 1) if H % d == 0]
    N = _log_int(rng, 1, 250)
    return {"op": op, "N": N, "H": H, "Hk": rng.choice(divs), "D": rng.choice([64, 128]),
            "gate": rng.choice([SCALAR, CHANNEL, SIGMOID]), "dtype": dtype, "pad": rng.choice([0, rng.randint(0, N - 1)])}


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

def _gate_inputs(rnd, case, dt, tokens, H, D):
    """The gate as the layer's projections give it, and the per-head parameters."""
    if case["gate"] == SCALAR:
        return {"g": (-0.1 * torch.nn.functional.softplus(rnd(tokens, H))).to(dt), "A_log": None, "dt_bias": None}
    return {"g": rnd(tokens, H, D).to(dt), "A_log": 1.5 * torch.rand(H, device=DEV, generator=rnd.gen),
            "dt_bias": 0.5 * rnd(H, D)}


def _rnd(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rnd(*shape):
        return torch.randn(shape, device=DEV, generator=gen)

    rnd.gen = gen
    return rnd


def prepare(case, seed):
    rnd, dt, s = _rnd(seed), _dtype(case), {"case": case}
    if case["op"] in ("scan_train", "scan_fwd"):
        H, D, lens = case["H"], case["D"], _lengths(case)
        tokens, N = sum(lens), len(lens)
        s["t"] = dict(_gate_inputs(rnd, case, dt, tokens, H, D), x=rnd(tokens, H, D).to(dt), h0=0.1 * rnd(N, H, D))
        if case["op"] == "scan_train":
            s["dy"], s["dht"] = rnd(tokens, H, D).to(dt), 0.1 * rnd(N, H, D)
        cu = np.concatenate([[0], np.cumsum(lens)])
        full = [n for n in range(N) if lens[n]]
        s["full"] = torch.tensor(full, device=DEV)
        s["first"] = torch.tensor([int(cu[n]) for n in full], device=DEV)
        s["last"] = torch.tensor([int(cu[n + 1]) - 1 for n in full], device=DEV)
        if own:
            from chunked_gated_delta_bwd_amd import binding as G
            s["prob"] = G.ScanProblem(case["B"], case["T"], H, D, N, case["gate"], G.GDR_BF16 if case["dtype"] == "bf16" else G.GDR_F32,
                                      cu_seqlens=cu.tolist() if case["seqs"] else None, gate_scale=GATE_SCALE,
                                      convex=case["convex"])
            s["ws"] = G.alloc_scan_workspace(s["prob"], DEV)
            s["y"], s["ht"] = torch.empty_like(s["t"]["x"]), torch.empty(N, H, D, device=DEV)
            if case["op"] == "scan_train":
                s["out"] = {"dx": torch.empty_like(s["t"]["x"]), "dg": torch.empty_like(s["t"]["g"]),
                            "dh0": torch.empty(N, H, D, device=DEV)}
                if case["gate"] != SCALAR:
                    s["out"].update(dA_log=torch.empty(H, device=DEV), ddt_bias=torch.empty(H, D, device=DEV))
    elif case["op"] == "scan_step":
        N, H, D = case["B"], case["H"], case["D"]
        s["t"] = dict(_gate_inputs(rnd, case, dt, N, H, D), x=rnd(N, H, D).to(dt), h0=None)
        _pool(s, rnd, N, N // 16, (H, D))
        s["y"] = torch.zeros(N, H, D, dtype=dt, device=DEV)
        if own:
            from chunked_gated_delta_bwd_amd import binding as G
            s["prob"] = G.ScanProblem(N, 1, H, D, N, case["gate"], G.GDR_BF16 if case["dtype"] == "bf16" else G.GDR_F32,
                                      gate_scale=GATE_SCALE, convex=case["convex"])
    elif case["op"] in ("norm_train", "norm_quant"):
        rows, width = case["rows"], case["width"]
        s["x"], s["w"] = rnd(rows, width).to(dt), 1.0 + 0.2 * rnd(width)
        s["res"] = (4.0 * rnd(rows, width)).to(dt) if case["res"] else None
        if case["op"] == "norm_train":
            s["dy"] = rnd(rows, width).to(dt)
            s["dres"] = rnd(rows, width).to(dt) if case["res"] else None
        if own:
            from chunked_gated_delta_bwd_amd import binding as G
            s["prob"] = G.NormProblem(rows, width, G.GDR_BF16 if case["dtype"] == "bf16" else G.GDR_F32, eps=EPS,
                                      group=case["group"])
            s["res_out"] = torch.empty_like(s["x"]) if case["res"] else None
            if case["op"] == "norm_train":
                s["y"], s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["x"]), torch.empty_like(s["w"])
                s["ws"] = G.alloc_norm_workspace(s["prob"], DEV)
            else:
                groups = -(-width // case["group"]) if case["group"] else 1
                s["q"] = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=DEV)
                s["scales"] = torch.empty(rows, groups, device=DEV)
    else:
        N, H, Hk, D = case["N"], case["H"], case["Hk"], case["D"]
        s["t"] = dict(_gate_inputs(rnd, case, dt, N, H, D), q=rnd(N, Hk, D).to(dt), k=rnd(N, Hk, D).to(dt),
                      v=rnd(N, H, D).to(dt), b=rnd(N, H).to(dt), h0=None)
        _pool(s, rnd, N, case["pad"], (H, D, D))
        s["o"] = torch.zeros(N, H, D, dtype=dt, device=DEV)
        if own:
            from chunked_gated_delta_bwd_amd import binding as G
            s["prob"] = G.Problem(N, 1, H, D, N, case["gate"], G.GDR_BF16 if case["dtype"] == "bf16" else G.GDR_F32,
                                  D ** -0.5, gate_scale=GATE_SCALE if case["gate"] == SIGMOID else 0.0, Hk=Hk)
    return s


def _pool(s, rnd, N, pad, shape):
    """A pool of states a little larger than the batch, the rows' slots in no order, the last `pad` rows without one."""
    s["state"] = 0.3 * rnd(N + 3, *shape)
    slots = torch.randperm(N + 3, device=DEV, generator=rnd.gen)[:N].to(torch.int32)
    slots[N - pad:] = -1
    s["slots"] = slots
    s["rows"] = torch.arange(N - pad, device=DEV)


# --------------------------------------------------------------------------------------------------------------
# the operators
# --------------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op in ("scan_train", "scan_fwd"):
        return _plain_scan(s, op == "scan_train")
    if op == "scan_step":
        return _plain_scan_step(s)
    if op == "norm_train":
        return _plain_norm(s)
    if op == "norm_quant":
        return _plain_norm_quant(s)
    return _plain_step(s)


def _run_own(s, op):
    from chunked_gated_delta_bwd_amd import binding as G
    if op in ("scan_train", "scan_fwd"):
        G.gdr_scan_fwd(s["prob"], s["t"], s["ws"], s["y"], ht=s["ht"])
        if op == "scan_fwd":
            return {"y": s["y"], "ht": s["ht"]}
        G.gdr_scan_bwd(s["prob"], s["t"], s["dy"], s["dht"], s["ws"], s["out"])
        return {"y": s["y"], "ht": s["ht"], **s["out"]}
    if op == "scan_step":
        G.gdr_scan_step(s["prob"], s["t"], s["state"], s["y"], slots=s["slots"])
        return {"y": s["y"], "state": s["state"]}
    if op == "norm_train":
        G.gdr_norm_fwd(s["prob"], s["x"], s["w"], s["y"], res=s["res"], res_out=s["res_out"])
        G.gdr_norm_bwd(s["prob"], s["x"] if s["res"] is None else s["res_out"], s["w"], s["dy"], s["dx"], s["dw"], s["ws"],
                       dres=s["dres"])
        out = {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    elif op == "norm_quant":
        G.gdr_norm_quant(s["prob"], s["x"], s["w"], s["q"], s["scales"], res=s["res"], res_out=s["res_out"])
        out = {"q": s["q"], "scales": s["scales"]}
    else:
        G.gdr_step(s["prob"], s["t"], s["state"], s["o"], slots=s["slots"])
        return {"o": s["o"], "state": s["state"]}
    return out if s["res"] is None else {**out, "res_out": s["res_out"]}


def _plain_log_decay(case, t):
    """lambda [tokens, H, D or 1] in 32 bits, and the pre-activation the gate's gradient needs."""
    g = t["g"].float()
    if case["gate"] == SCALAR:
        return g[..., None], None
    z, eA = g + t["dt_bias"], t["A_log"].exp()[:, None]
    if case["gate"] == CHANNEL:
        return -eA * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))), z
    return GATE_SCALE / (1 + torch.exp(-eA * z)), z


def _linear_scan(a, u):
    """s_t = a_t s_{t-1} + u_t over the first axis from s = 0, by doubling."""
    d, T = 1, u.shape[0]
    while d < T:
        u = torch.cat([u[:d], u[d:] + a[d:] * u[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return u


def _plain_scan(s, train):
    case, t = s["case"], s["t"]
    x = t["x"].float()
    lam, z = _plain_log_decay(case, t)
    a = torch.exp(lam).expand_as(x)
    u = -torch.expm1(lam) * x if case["convex"] else x.clone()
    first, last, full, h0 = s["first"], s["last"], s["full"], t["h0"]
    u[first] += a[first] * h0[full]
    cut = a.clone()
    cut[first] = 0
    st = _linear_scan(cut, u)
    ht = h0.clone()
    ht[full] = st[last]
    y = st.to(t["x"].dtype)
    if not train:
        return {"y": y, "ht": ht}
    dy = s["dy"].to(torch.float32, copy=True)
    dy[last] += s["dht"][full]
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]
    nxt[last] = 0
    ds = _linear_scan(nxt.flip(0), dy.flip(0)).flip(0)
    prev = torch.zeros_like(st)
    prev[1:] = st[:-1]
    prev[first] = h0[full]
    dx = -torch.expm1(lam) * ds if case["convex"] else ds
    dlam = a * ds * (prev - x if case["convex"] else prev)
    dh0 = s["dht"].clone()
    dh0[full] = (a * ds)[first]
    out = {"y": y, "ht": ht, "dx": dx.to(y.dtype), "dh0": dh0}
    if case["gate"] == SCALAR:
        out["dg"] = dlam.sum(-1).to(y.dtype)
        return out
    eA = t["A_log"].exp()[:, None]
    if case["gate"] == CHANNEL:
        dz, dA = dlam * (-eA / (1 + torch.exp(-z))), dlam * lam
    else:
        p = 1 / (1 + torch.exp(-eA * z))
        dz = dlam * (GATE_SCALE * p * (1 - p) * eA)
        dA = dz * z
    out.update(dg=dz.to(y.dtype), dA_log=dA.sum((0, 2), dtype=torch.float64).float(),
               ddt_bias=dz.sum(0, dtype=torch.float64).float())
    return out


def _plain_scan_step(s):
    case, t, rows = s["case"], s["t"], s["rows"]
    lam, _ = _plain_log_decay(case, t)
    x = t["x"].float()
    u = -torch.expm1(lam) * x if case["convex"] else x
    slots = s["slots"][rows].long()
    new = torch.exp(lam[rows]) * s["state"][slots] + u[rows]
    s["state"][slots] = new
    s["y"][rows] = new.to(s["y"].dtype)
    return {"y": s["y"], "state": s["state"]}


def _plain_norm(s):
    x, w = s["x"].float(), s["w"]
    r = x if s["res"] is None else x + s["res"].float()
    out = {"y": (r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * w).to(s["x"].dtype)}
    if s["res"] is not None:
        out["res_out"] = r.to(s["x"].dtype)
        r = out["res_out"].float()
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    dy, n = s["dy"].float(), r * rstd
    dn = dy * w
    dx = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out.update(dx=dx.to(s["x"].dtype), dw=(dy * n).sum(0, dtype=torch.float64).float())
    return out


def _plain_norm_quant(s):
    case = s["case"]
    r = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["w"]
    rows, width = y.shape
    group = case["group"] or width
    groups = -(-width // group)
    y = torch.nn.functional.pad(y, (0, groups * group - width)).view(rows, groups, group)
    scales = (y.abs().amax(-1) / 448.0).clamp(min=2.0 ** -126)
    q = (y / scales[..., None]).clamp(-448.0, 448.0).view(rows, groups * group)[:, :width]
    out = {"q": q.to(torch.float8_e4m3fn), "scales": scales}
    if s["res"] is not None:
        out["res_out"] = r.to(s["x"].dtype)
    return out


def _plain_step(s):
    case, t, rows = s["case"], s["t"], s["rows"]
    H, Hk = case["H"], case["Hk"]
    q, k = t["q"].float(), t["k"].float()
    q = (q * torch.rsqrt(q.square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(H // Hk, 1)[rows]
    k = (k * torch.rsqrt(k.square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(H // Hk, 1)[rows]
    lam, _ = _plain_log_decay(case, t)
    beta = 1 / (1 + torch.exp(-t["b"].float()[rows]))
    slots = s["slots"][rows].long()
    st = s["state"][slots] * torch.exp(lam[rows])[:, :, None, :]
    d = beta[..., None] * (t["v"].float()[rows] - (st * k[:, :, None, :]).sum(-1))
    st = st + d[..., None] * k[:, :, None, :]
    s["state"][slots] = st
    s["o"][rows] = ((st * q[:, :, None, :]).sum(-1) * case["D"] ** -0.5).to(s["o"].dtype)
    return {"o": s["o"], "state": s["state"]}


# --------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("scan_train", "scan_fwd"):
        lens = _lengths(case)
        el, st = sum(lens) * case["H"] * case["D"], len(lens) * case["H"] * case["D"]
        g = sum(lens) * case["H"] if case["gate"] == SCALAR else el
        par = 0 if case["gate"] == SCALAR else 4 * (case["H"] + case["H"] * case["D"])
        if op == "scan_fwd":
            return {"bytes": e * (2 * el + g) + 8 * st + par, "flops": 4 * el}
        return {"bytes": e * (4 * el + 2 * g) + 16 * st + 2 * par, "flops": 14 * el}
    if op == "scan_step":
        N, C = case["B"], case["H"] * case["D"]
        on = (N - N // 16) * C
        g = N * case["H"] if case["gate"] == SCALAR else on
        par = 0 if case["gate"] == SCALAR else 4 * (case["H"] + C)
        return {"bytes": e * (2 * on + g) + 8 * on + 4 * N + par, "flops": 4 * on}
    if op.startswith("norm"):
        el, w = case["rows"] * case["width"], case["width"]
        if op == "norm_train":
            return {"bytes": e * el * (7 if case["res"] else 4) + 8 * w, "flops": 16 * el}
        groups = -(-w // case["group"]) if case["group"] else 1
        return {"bytes": el * (e * (3 if case["res"] else 1) + 1) + 4 * case["rows"] * groups + 4 * w, "flops": 8 * el}
    on, H, Hk, D = case["N"] - case["pad"], case["H"], case["Hk"], case["D"]
    g = on * H * (1 if case["gate"] == SCALAR else D)
    par = 0 if case["gate"] == SCALAR else 4 * (H + H * D)
    return {"bytes": 8 * on * H * D * D + e * (on * (2 * Hk * D + 2 * H * D + H) + g) + 4 * case["N"] + par,
            "flops": 7 * on * H * D * D}


# --------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, token by token
# --------------------------------------------------------------------------------------------------------------

def _exact_gate(case, t):
    g = t["g"].double()
    if case["gate"] == SCALAR:
        return g.unsqueeze(-1), None, None
    A, z = t["A_log"].double().view(1, -1, 1), g + t["dt_bias"].double()
    if case["gate"] == CHANNEL:
        lam = -A.exp() * torch.logaddexp(z, torch.zeros_like(z))
        return lam, -A.exp() * torch.sigmoid(z), lam                       # lambda, d lambda/d z, d lambda/d A_log
    w = A.exp() * z
    slope = GATE_SCALE * torch.sigmoid(w) * torch.sigmoid(-w)
    return GATE_SCALE * torch.sigmoid(w), slope * A.exp(), slope * w


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("scan_train", "scan_fwd"):
        return _exact_scan(case, s)
    if case["op"] == "scan_step":
        lam, _, _ = _exact_gate(case, s["t"])
        a, x, st, y = lam.exp(), s["t"]["x"].double(), s["state"].double(), s["y"].double()
        on = s["rows"].numel()
        at = s["slots"][:on].long()
        st[at] = a[:on] * st[at] + ((1 - a) * x if case["convex"] else x)[:on]
        y[:on] = st[at]
        return {"y": y, "state": st}
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    return _exact_step(case, s)


def _exact_scan(case, s):
    t, lens, train = s["t"], _lengths(case), case["op"] == "scan_train"
    lam, dz, dA = _exact_gate(case, t)
    x, a, h0 = t["x"].double(), lam.exp(), t["h0"].double()
    m = -torch.expm1(lam) if case["convex"] else torch.ones_like(lam)
    before, y, ht = torch.empty_like(x), torch.empty_like(x), h0.clone()
    at = 0
    for n, L in enumerate(lens):
        st = h0[n]
        for i in range(at, at + L):
            before[i] = st
            st = torch.addcmul(m[i] * x[i], a[i], st)
            y[i] = st
        ht[n] = st
        at += L
    if not train:
        return {"y": y, "ht": ht}
    dy, ds, dh0 = s["dy"].double(), torch.empty_like(x), s["dht"].double()
    at = sum(lens)
    for n in range(len(lens) - 1, -1, -1):
        e = dh0[n].clone()
        for i in range(at - 1, at - 1 - lens[n], -1):
            e = e + dy[i]
            ds[i] = e
            e = a[i] * e
        dh0[n] = e
        at -= lens[n]
    # d u/d lambda of the convex input is -a x
    dlam = ds * a * (before - x) if case["convex"] else ds * a * before
    out = {"y": y, "ht": ht, "dx": m * ds, "dh0": dh0}
    if dz is None:
        return {**out, "dg": dlam.sum(-1)}
    return {**out, "dg": dlam * dz, "ddt_bias": (dlam * dz).sum(0), "dA_log": (dlam * dA).sum(0).sum(-1)}


def _exact_norm(case, s):
    w = s["w"].double()
    r = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
    y = r / (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
    out = {} if s["res"] is None else {"res_out": r}
    if case["op"] == "norm_quant":
        scales = torch.stack([c.abs().amax(-1) for c in y.split(case["group"] or case["width"], -1)], -1) / 448
        scales = scales.clamp(min=2.0 ** -126)
        q = torch.cat([c / scales[:, i:i + 1] for i, c in enumerate(y.split(case["group"] or case["width"], -1))], -1)
        return {**out, "q": q, "scales": scales}
    if s["res"] is not None:
        r = r.to(s["x"].dtype).double()                  # the backward reads the residual as it was stored
    rms, dy = (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt(), s["dy"].double()
    # y_i = w_i r_i / rms, d rms/d r_j = r_j / (width rms)
    dx = w * dy / rms - r * (w * dy * r).sum(-1, keepdim=True) / (case["width"] * rms.pow(3))
    if s["dres"] is not None:
        dx = dx + s["dres"].double()
    return {**out, "y": y, "dx": dx, "dw": (dy * r / rms).sum(0)}


def _exact_step(case, s):
    t, H, Hk, D = s["t"], case["H"], case["Hk"], case["D"]
    on = s["rows"].numel()
    head = torch.arange(H, device=DEV) // (H // Hk)
    q, k = t["q"].double()[:on, head], t["k"].double()[:on, head]
    q, k = q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt(), k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    a, beta = _exact_gate(case, t)[0][:on].exp().expand(on, H, D), torch.sigmoid(t["b"].double()[:on])
    # S <- S Diag(a) (I - beta k k^T) + beta v k^T
    kk = beta[..., None, None] * k[..., :, None] * k[..., None, :]
    move = a[..., :, None] * (torch.eye(D, device=DEV, dtype=torch.float64) - kk)
    at, st, o = s["slots"][:on].long(), s["state"].double(), s["o"].double()
    st[at] = st[at] @ move + beta[..., None, None] * t["v"].double()[:on, :, :, None] * k[..., None, :]
    o[:on] = D ** -0.5 * (st[at] @ q[..., None])[..., 0]
    return {"o": o, "state": st}
