"""Checks of the operators around the delta rule that need no GPU: the C ABI's
refusals (every case fails validation, so no HIP call is made), the binding's
refusals of tensors of another type, size, layout or device, and workspace sizes."""

import ctypes
import os

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not os.path.exists(B.library_path()):
        from chunked_gated_delta_bwd_amd import build
        build.build()
    B.load_library()


def refused(status, text, fn, *args, **kw):
    with pytest.raises(B.GdrError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)
    assert text in str(e.value), str(e.value)


def call(name, *args):
    """The library's own function with made-up addresses."""
    B._check(getattr(B.load_library(), name)(*args))


def scan(**kw):
    args = dict(B=1, T=300, H=2, D=64, N=1, gate=0, dtype=B.GDR_BF16)
    args.update(kw)
    return B.ScanProblem(**args)


@pytest.mark.parametrize("kw,status,text", [
    (dict(D=0), B.GDR_EINVAL, "bad B/T/H/D/N"),
    (dict(D=12), B.GDR_EUNSUPPORTED, "multiple of 8"),
    (dict(D=264), B.GDR_EUNSUPPORTED, "multiple of 8"),
    (dict(H=0), B.GDR_EINVAL, "bad"),
    (dict(T=-1), B.GDR_EINVAL, "bad"),
    (dict(gate=3), B.GDR_EINVAL, "unknown gate"),
    (dict(gate=2, gate_scale=0.5), B.GDR_EINVAL, "gate_scale"),
    (dict(gate=2, gate_scale=float("nan")), B.GDR_EINVAL, "gate_scale"),
    (dict(dtype=7), B.GDR_EINVAL, "unknown dtype"),
    (dict(convex=2), B.GDR_EINVAL, "convex"),
    (dict(N=2), B.GDR_EINVAL, "N == B"),
    (dict(B=2, N=2, cu_seqlens=[0, 100, 300]), B.GDR_EINVAL, "B == 1"),
    (dict(N=2, cu_seqlens=[0, 100, 90]), B.GDR_EINVAL, "decreases"),
    (dict(N=2, cu_seqlens=[0, 100, 200]), B.GDR_EINVAL, "!= T"),
    (dict(N=2, cu_seqlens=[0, 1 << 40, 1 << 41]), B.GDR_EINVAL, "> T"),
    (dict(N=1, cu_seqlens=[3, 300]), B.GDR_EINVAL, "expected 0"),
    (dict(H=1 << 20, D=256), B.GDR_EUNSUPPORTED, "too large"),
    (dict(B=1 << 20, N=1 << 20, T=1 << 12), B.GDR_EUNSUPPORTED, "too large"),
])
def test_scan_shape_validation(kw, status, text):
    refused(status, text, B.gdr_scan_workspace_bytes, scan(**kw))


def test_cu_seqlens_of_another_length_are_refused():
    refused(B.GDR_EINVAL, "cu_seqlens has 2 entries", scan, N=2, cu_seqlens=[0, 300])


def test_scan_workspace_grows_with_tiles():
    a, b, c = (B.gdr_scan_workspace_bytes(scan(T=t)) for t in (128, 129, 256))
    assert 0 < a < b == c
    assert B.gdr_scan_workspace_bytes(scan(T=300, N=4, cu_seqlens=[0, 1, 1, 130, 300])) > B.gdr_scan_workspace_bytes(scan())
    assert B.gdr_scan_workspace_bytes(scan(gate=1)) > B.gdr_scan_workspace_bytes(scan())


X, G, A, DTB, H0, Y, WS = (0x100000 * i for i in range(1, 8))


def scan_call(which, prob, x=X, g=G, A_log=None, dt_bias=None, h0=None, y=Y, ht=None, ws=WS, ws_bytes=None, dy=Y, dht=None,
              dx=0x900000, dg=0xa00000, dh0=None, dA=None, ddt=None, state=0xb00000, P=4, slots=None, null=None):
    n = B.gdr_scan_workspace_bytes(prob) if ws_bytes is None else ws_bytes
    inp = None if null == "in" else ctypes.byref(B.ScanInputs(x, g, A_log, dt_bias, h0))
    if which == "fwd":
        call("gdr_scan_fwd", prob.ref, inp, ws, n, y, ht, None)
    elif which == "bwd":
        gr = None if null == "grads" else ctypes.byref(B.ScanGrads(dx, dg, dh0, dA, ddt))
        call("gdr_scan_bwd", prob.ref, inp, dy, dht, ws, n, gr, None)
    else:
        call("gdr_scan_step", prob.ref, inp, state, P, slots, y, None)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status,text", [
    (dict(null="in"), B.GDR_EINVAL, "inputs is NULL"),
    (dict(x=None), B.GDR_EINVAL, "input x is NULL"),
    (dict(g=G + 8), B.GDR_EINVAL, "input g is not 16-byte aligned"),
    (dict(h0=H0 + 4), B.GDR_EINVAL, "h0 is not 16-byte"),
    (dict(A_log=A, dt_bias=DTB), B.GDR_EINVAL, "takes no A_log"),
    (dict(ws=None), B.GDR_EINVAL, "workspace is NULL"),
    (dict(ws=WS + 16), B.GDR_EINVAL, "256-byte aligned"),
    (dict(ws_bytes=256), B.GDR_EWORKSPACE, "workspace 256 bytes"),
])
def test_scan_refusals(which, kw, status, text):
    refused(status, text, scan_call, which, scan(), **kw)


@pytest.mark.parametrize("which,kw,text", [
    ("fwd", dict(y=None), "y is NULL"),
    ("fwd", dict(y=Y + 2), "y is not 16-byte"),
    ("fwd", dict(ht=Y + 4), "ht is not 16-byte"),
    ("bwd", dict(null="grads"), "grads is NULL"),
    ("bwd", dict(dy=None), "dy is NULL"),
    ("bwd", dict(dx=None), "output dx is NULL"),
    ("bwd", dict(dg=None), "output dg is NULL"),
    ("bwd", dict(dht=Y + 4), "dht is not"),
    ("bwd", dict(dh0=Y + 4), "dh0 is not"),
    ("bwd", dict(dA=A), "scalar gate has no dA_log"),
])
def test_scan_output_refusals(which, kw, text):
    refused(B.GDR_EINVAL, text, scan_call, which, scan(), **kw)


def test_scan_per_channel_parameters_are_required():
    p = scan(gate=1)
    refused(B.GDR_EINVAL, "needs A_log and dt_bias", scan_call, "fwd", p, A_log=A)
    refused(B.GDR_EINVAL, "dA_log is NULL", scan_call, "bwd", p, A_log=A, dt_bias=DTB)


@pytest.mark.parametrize("shape,kw,text", [
    (dict(T=2), {}, "T == 1"),
    (dict(T=1, N=1, cu_seqlens=[0, 1]), {}, "T == 1"),
    (dict(T=1), dict(h0=H0), "not from h0"),
    (dict(T=1), dict(x=None), "input x"),
    (dict(T=1), dict(y=None), "y is NULL"),
    (dict(T=1), dict(state=None), "state is NULL"),
    (dict(T=1), dict(state=0xb00004), "state is not 16-byte"),
    (dict(T=1), dict(P=-1), "P (-1)"),
    (dict(T=1, B=5, N=5), dict(P=4), "as many states"),
    (dict(T=1), dict(slots=0xc00002), "slots is not 4-byte"),
])
def test_scan_step_refusals(shape, kw, text):
    refused(B.GDR_EINVAL, text, scan_call, "step", scan(**shape), **kw)


def step_call(prob, state=0xb00000, P=4, slots=None, o=Y, h0=None, q=X):
    inp = B.Inputs(q, X, X, G, G, None, None, h0)
    call("gdr_step", ctypes.byref(prob.shape), ctypes.byref(inp), state, P, slots, o, None)


@pytest.mark.parametrize("shape,kw,status,text", [
    (dict(T=2), {}, B.GDR_EINVAL, "T == 1"),
    (dict(cu_seqlens=[0, 1]), {}, B.GDR_EINVAL, "T == 1"),
    (dict(D=96), {}, B.GDR_EUNSUPPORTED, "head dim"),
    (dict(H=4, Hk=3), {}, B.GDR_EINVAL, "Hk"),
    ({}, dict(h0=H0), B.GDR_EINVAL, "not from h0"),
    ({}, dict(q=None), B.GDR_EINVAL, "input q"),
    ({}, dict(o=None), B.GDR_EINVAL, "o is NULL"),
    ({}, dict(o=Y + 8), B.GDR_EINVAL, "o is not"),
    ({}, dict(state=None), B.GDR_EINVAL, "state is NULL"),
    ({}, dict(P=-3), B.GDR_EINVAL, "P (-3)"),
    (dict(B=9, N=9), {}, B.GDR_EINVAL, "as many states"),
    ({}, dict(slots=0xc00001), B.GDR_EINVAL, "slots"),
    (dict(gate=1), {}, B.GDR_EINVAL, "needs A_log"),
])
def test_step_refusals(shape, kw, status, text):
    args = dict(B=1, T=1, H=2, D=64, N=1, gate=0, dtype=0, scale=1.0)
    args.update(shape)
    refused(status, text, step_call, B.Problem(**args), **kw)


def norm_call(which, prob, x=X, res=None, w=A, y=Y, q=Y, scales=H0, res_out=None, dy=Y, dres=None, ws=WS, ws_bytes=None,
              dx=0x900000, dw=0xa00000):
    if which == "fwd":
        call("gdr_norm_fwd", prob.ref, x, res, w, y, res_out, None)
    elif which == "quant":
        call("gdr_norm_quant", prob.ref, x, res, w, q, scales, res_out, None)
    else:
        n = B.gdr_norm_workspace_bytes(prob) if ws_bytes is None else ws_bytes
        call("gdr_norm_bwd", prob.ref, x, w, dy, dres, ws, n, dx, dw, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(rows=-1), B.GDR_EINVAL, "bad rows/width"),
    (dict(width=0), B.GDR_EINVAL, "bad rows/width"),
    (dict(width=32769), B.GDR_EUNSUPPORTED, "width"),
    (dict(rows=1 << 31), B.GDR_EUNSUPPORTED, "rows"),
    (dict(dtype=2), B.GDR_EINVAL, "dtype"),
    (dict(eps=-1.0), B.GDR_EINVAL, "eps"),
    (dict(eps=float("nan")), B.GDR_EINVAL, "eps"),
    (dict(eps=float("inf")), B.GDR_EINVAL, "eps"),
])
def test_norm_shape_validation(kw, status, text):
    args = dict(rows=4, width=128, dtype=0)
    args.update(kw)
    p = B.NormProblem(**args)
    refused(status, text, B.gdr_norm_workspace_bytes, p)
    for which in ("fwd", "quant"):
        refused(status, text, norm_call, which, p)
    refused(status, text, norm_call, "bwd", p, ws_bytes=1 << 30)


@pytest.mark.parametrize("which,kw,status,text", [
    ("fwd", dict(x=None), B.GDR_EINVAL, "x is NULL"),
    ("fwd", dict(y=None), B.GDR_EINVAL, "y is NULL"),
    ("fwd", dict(y=Y + 8), B.GDR_EINVAL, "y is not"),
    ("fwd", dict(w=A + 4), B.GDR_EINVAL, "w is not"),
    ("fwd", dict(res=X), B.GDR_EINVAL, "go together"),
    ("fwd", dict(res_out=X), B.GDR_EINVAL, "go together"),
    ("fwd", dict(res=X, res_out=Y), B.GDR_EINVAL, "same tensor"),
    ("quant", dict(q=None), B.GDR_EINVAL, "q is NULL"),
    ("quant", dict(scales=None), B.GDR_EINVAL, "scales is NULL"),
    ("quant", dict(scales=H0 + 4), B.GDR_EINVAL, "scales is not"),
    ("quant", dict(res=X), B.GDR_EINVAL, "go together"),
    ("bwd", dict(x=None), B.GDR_EINVAL, "r is NULL"),
    ("bwd", dict(dy=None), B.GDR_EINVAL, "dy is NULL"),
    ("bwd", dict(dx=None), B.GDR_EINVAL, "dx is NULL"),
    ("bwd", dict(dres=X + 8), B.GDR_EINVAL, "dres is not"),
    ("bwd", dict(ws=None), B.GDR_EINVAL, "workspace is NULL"),
    ("bwd", dict(ws=WS + 64), B.GDR_EINVAL, "256-byte"),
    ("bwd", dict(ws_bytes=16), B.GDR_EWORKSPACE, "workspace 16 bytes"),
])
def test_norm_refusals(which, kw, status, text):
    refused(status, text, norm_call, which, B.NormProblem(4, 128, B.GDR_BF16), **kw)


def test_norm_group_refusal():
    refused(B.GDR_EUNSUPPORTED, "group 64", norm_call, "quant", B.NormProblem(4, 128, B.GDR_BF16, group=64))


# ---- the binding's own checks (CPU tensors: a call that passed the others is
# refused for its device, so nothing here reaches the library) ----

def test_binding_checks_tensors():
    p = B.NormProblem(4, 64, B.GDR_BF16)
    x, w, y = torch.zeros(4, 64, dtype=BF), torch.zeros(64), torch.zeros(4, 64, dtype=BF)
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_norm_fwd, p, x, w, y)
    refused(B.GDR_EINVAL, "x is torch.float32", B.gdr_norm_fwd, p, x.float(), w, y)
    refused(B.GDR_EINVAL, "w is torch.bfloat16", B.gdr_norm_fwd, p, x, w.to(BF), y)
    refused(B.GDR_EINVAL, "y has 192 elements", B.gdr_norm_fwd, p, x, w, y[:3])
    refused(B.GDR_EINVAL, "x is not contiguous", B.gdr_norm_fwd, p, torch.zeros(64, 4, dtype=BF).t(), w, y)
    refused(B.GDR_EINVAL, "q is torch.uint8", B.gdr_norm_quant, p, x, w, torch.zeros(4, 64, dtype=torch.uint8),
            torch.zeros(4, 1))
    refused(B.GDR_EINVAL, "scales has 8 elements", B.gdr_norm_quant, p, x, w, torch.zeros(4, 64).to(E4), torch.zeros(4, 2))
    refused(B.GDR_EINVAL, "dw has 4 elements", B.gdr_norm_bwd, p, x, w, y, y, torch.zeros(4), None)
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_norm_bwd, p, x, w, y, y, w, None)


def test_binding_checks_scan_tensors():
    p = scan(T=3, gate=1)
    t = {"x": torch.zeros(3, 2, 64, dtype=BF), "g": torch.zeros(3, 2, 64, dtype=BF), "A_log": torch.zeros(2),
         "dt_bias": torch.zeros(2, 64), "h0": torch.zeros(1, 2, 64)}
    y, ws = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(1 << 16, dtype=torch.uint8)
    out = {"dx": y, "dg": y, "dA_log": t["A_log"], "ddt_bias": t["dt_bias"]}
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_scan_fwd, p, t, ws, y)
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_scan_bwd, p, t, y, None, ws, out)
    refused(B.GDR_EINVAL, "g has 6 elements", B.gdr_scan_fwd, p, {**t, "g": torch.zeros(3, 2, dtype=BF)}, ws, y)
    refused(B.GDR_EINVAL, "h0 has 64", B.gdr_scan_fwd, p, {**t, "h0": torch.zeros(64)}, ws, y)
    refused(B.GDR_EINVAL, "ht is torch.bfloat16", B.gdr_scan_fwd, p, t, ws, y, ht=torch.zeros(1, 2, 64, dtype=BF))
    refused(B.GDR_EINVAL, "dht has 2", B.gdr_scan_bwd, p, t, y, torch.zeros(2), ws, out)
    refused(B.GDR_EINVAL, "ddt_bias has 2", B.gdr_scan_bwd, p, t, y, None, ws, {**out, "ddt_bias": torch.zeros(2)})
    one = scan(T=1, B=3, N=3)
    t1 = {"x": t["x"], "g": torch.zeros(3, 2, dtype=BF), "h0": None}
    st = torch.zeros(5, 2, 64)
    refused(B.GDR_EINVAL, "state has shape", B.gdr_scan_step, one, t1, torch.zeros(5, 64), y)
    refused(B.GDR_EINVAL, "state is torch.bfloat16", B.gdr_scan_step, one, t1, st.to(BF), y)
    refused(B.GDR_EINVAL, "slots is torch.int64", B.gdr_scan_step, one, t1, st, y, slots=torch.zeros(3, dtype=torch.int64))
    refused(B.GDR_EINVAL, "slots has 2", B.gdr_scan_step, one, t1, st, y, slots=torch.zeros(2, dtype=torch.int32))
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_scan_step, one, t1, st, y)


def test_binding_checks_step_tensors():
    p = B.Problem(3, 1, 4, 64, 3, 0, B.GDR_F32, 1.0, Hk=2)
    t = {"q": torch.zeros(3, 2, 64), "k": torch.zeros(3, 2, 64), "v": torch.zeros(3, 4, 64), "g": torch.zeros(3, 4),
         "b": torch.zeros(3, 4)}
    st, o = torch.zeros(3, 4, 64, 64), torch.zeros(3, 4, 64)
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_step, p, t, st, o)
    refused(B.GDR_EINVAL, "q has 768", B.gdr_step, p, {**t, "q": t["v"]}, st, o)
    refused(B.GDR_EINVAL, "g has 768", B.gdr_step, p, {**t, "g": t["v"]}, st, o)
    refused(B.GDR_EINVAL, "o is torch.bfloat16", B.gdr_step, p, t, st, o.to(BF))
    refused(B.GDR_EINVAL, "state is not contiguous", B.gdr_step, p, t, st.transpose(2, 3), o)
    refused(B.GDR_EINVAL, "slots has 4", B.gdr_step, p, t, st, o, slots=torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("kw,fits", [
    (dict(T=1, D=1, H=64, B=(1 << 24) - 1, N=(1 << 24) - 1), True),
    (dict(T=1, D=1, H=64, B=1 << 24, N=1 << 24), False),
    (dict(T=64, D=128, H=32, B=(1 << 18) - 1, N=(1 << 18) - 1, gate=1), True),
    (dict(T=64, D=128, H=32, B=1 << 18, N=1 << 18, gate=1), False),
])
def test_scan_launches_under_two_to_the_32_threads(kw, fits):
    """256 threads a tile: 2^24 tiles are one launch too many."""
    if fits:
        assert B.gdr_scan_workspace_bytes(scan(**kw)) > 0
    else:
        refused(B.GDR_EUNSUPPORTED, "too large", B.gdr_scan_workspace_bytes, scan(**kw))


@pytest.mark.parametrize("width,dtype,rows", [
    (32768, B.GDR_BF16, 1 << 22),    # 1024 threads a row
    (4100, B.GDR_F32, 1 << 22),
    (8192, B.GDR_BF16, 1 << 24),     # 256
    (2048, B.GDR_BF16, 1 << 26),     # 64
])
def test_norm_launches_under_two_to_the_32_threads(width, dtype, rows):
    assert B.gdr_norm_workspace_bytes(B.NormProblem(rows - 4, width, dtype)) > 0
    refused(B.GDR_EUNSUPPORTED, "too many rows", B.gdr_norm_workspace_bytes, B.NormProblem(rows, width, dtype))


def test_step_launches_under_two_to_the_32_threads():
    """128 / 32 workgroups of 256 threads a row and head; 2^22 rows and heads are too many."""
    n = 1 << 18
    prob = B.Problem(B=n, T=1, H=16, D=128, N=n, gate=0, dtype=B.GDR_BF16, scale=1.0)
    refused(B.GDR_EUNSUPPORTED, "too many rows", step_call, prob)
