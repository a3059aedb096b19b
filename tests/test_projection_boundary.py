"""Checks of linear attention with a decay for each head, of the e4m3 product and of its
quantisation that need no GPU: the C ABI's refusals (every case fails validation, so no HIP
call is made), the largest shapes on both sides, the binding's refusals of tensors of
another type, size, layout or device, and workspace sizes."""

import ctypes
import os

import pytest
import torch

from chunked_gated_delta_bwd_amd import binding as B

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
X, L, H0, Y, WS = (0x100000 * i for i in range(1, 6))


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


# ---- linear attention ----

def lin(**kw):
    args = dict(B=1, T=300, H=2, D=64, N=1, dtype=B.GDR_BF16, scale=1.0)
    args.update(kw)
    return B.LinProblem(**args)


def lin_call(which, prob, q=X, k=X, v=X, decay=L, h0=None, ws=WS, ws_bytes=None, o=Y, ht=None, dO=Y, dht=None, dq=0x900000,
             dk=0xa00000, dv=0xb00000, dh0=None, state=0xc00000, P=4, slots=None, null=None):
    n = (1 << 30) if ws_bytes is None else ws_bytes
    inp = None if null == "in" else ctypes.byref(B.LinInputs(q, k, v, decay, h0))
    if which == "fwd":
        call("gdr_lin_fwd", prob.ref, inp, ws, n, o, ht, None)
    elif which == "bwd":
        gr = None if null == "grads" else ctypes.byref(B.LinGrads(dq, dk, dv, dh0))
        call("gdr_lin_bwd", prob.ref, inp, dO, dht, ws, n, gr, None)
    else:
        call("gdr_lin_step", prob.ref, inp, state, P, slots, o, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=2), B.GDR_EINVAL, "dtype"),
    (dict(H=0), B.GDR_EINVAL, "bad B/T/H/D/N"),
    (dict(T=-1), B.GDR_EINVAL, "bad B/T/H/D/N"),
    (dict(D=0), B.GDR_EINVAL, "bad B/T/H/D/N"),
    (dict(D=96), B.GDR_EUNSUPPORTED, "head dim 96"),
    (dict(D=256), B.GDR_EUNSUPPORTED, "head dim 256"),
    (dict(H=4, Hk=3), B.GDR_EINVAL, "Hk 3"),
    (dict(H=2, Hk=4), B.GDR_EINVAL, "Hk 4"),
    (dict(Hk=-1), B.GDR_EINVAL, "Hk -1"),
    (dict(scale=float("nan")), B.GDR_EINVAL, "finite"),
    (dict(scale=float("inf")), B.GDR_EINVAL, "finite"),
    (dict(N=2), B.GDR_EINVAL, "N == B"),
    (dict(B=2, N=2, cu_seqlens=[0, 5, 300]), B.GDR_EINVAL, "B == 1"),
    (dict(N=0, cu_seqlens=[0]), B.GDR_EINVAL, "N >= 1"),
    (dict(cu_seqlens=[1, 300]), B.GDR_EINVAL, "cu_seqlens[0]"),
    (dict(N=2, cu_seqlens=[0, 200, 100]), B.GDR_EINVAL, "decreases at 1"),
    (dict(N=2, cu_seqlens=[0, 301, 301]), B.GDR_EINVAL, "> T = 300"),
    (dict(N=2, cu_seqlens=[0, 100, 200]), B.GDR_EINVAL, "!= T = 300"),
    (dict(H=(1 << 16) + 1, T=1), B.GDR_EUNSUPPORTED, "too large"),
])
def test_lin_shape_validation(kw, status, text):
    p = lin(**kw)
    refused(status, text, B.gdr_lin_workspace_bytes, p)
    refused(status, text, B.gdr_lin_workspace_bytes, p, True)
    for which in ("fwd", "bwd", "step"):
        refused(status, text, lin_call, which, p)


@pytest.mark.parametrize("kw,fits", [
    (dict(H=1, T=(1 << 26) - 65), True),                    # 2^20 - 2 blocks and a sequence
    (dict(H=1, T=(1 << 26) - 64), False),
    (dict(H=1 << 16, T=1, B=15, N=15), True),               # 15 blocks of 2^16 heads
    (dict(H=1 << 16, T=1, B=16, N=16), False),
    (dict(H=1, T=1, B=(1 << 20) - (1 << 14) - 1, N=(1 << 20) - (1 << 14) - 1), True),
    (dict(H=1, T=0, B=1 << 20, N=1 << 20), False),
    (dict(H=2, T=(1 << 31) - 1, B=(1 << 31) - 1, N=(1 << 31) - 1), False),   # 2^62 tokens
])
def test_the_largest_attentions(kw, fits):
    p = lin(**kw)
    if fits:
        assert B.gdr_lin_workspace_bytes(p, True) >= 0
    else:
        refused(B.GDR_EUNSUPPORTED, "too large", B.gdr_lin_workspace_bytes, p)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status,text", [
    (dict(null="in"), B.GDR_EINVAL, "inputs is NULL"),
    (dict(q=None), B.GDR_EINVAL, "input q is NULL"),
    (dict(k=X + 8), B.GDR_EINVAL, "input k is not 16-byte"),
    (dict(v=None), B.GDR_EINVAL, "input v is NULL"),
    (dict(decay=None), B.GDR_EINVAL, "log_decay is NULL"),
    (dict(decay=L + 4), B.GDR_EINVAL, "log_decay is not"),
    (dict(h0=H0 + 4), B.GDR_EINVAL, "h0 is not 16-byte"),
    (dict(ws=None), B.GDR_EINVAL, "workspace is NULL"),
    (dict(ws=WS + 16), B.GDR_EINVAL, "256-byte aligned"),
    (dict(ws_bytes=256), B.GDR_EWORKSPACE, "workspace 256 bytes"),
])
def test_lin_refusals(which, kw, status, text):
    refused(status, text, lin_call, which, lin(T=30000), **kw)


@pytest.mark.parametrize("which,kw,text", [
    ("fwd", dict(o=None), "o is NULL"),
    ("fwd", dict(o=Y + 2), "o is not 16-byte"),
    ("fwd", dict(ht=Y + 4), "ht is not 16-byte"),
    ("bwd", dict(null="grads"), "grads is NULL"),
    ("bwd", dict(dO=None), "dO is NULL"),
    ("bwd", dict(dq=None), "output dq is NULL"),
    ("bwd", dict(dk=None), "output dk is NULL"),
    ("bwd", dict(dv=Y + 8), "output dv is not"),
    ("bwd", dict(dht=Y + 4), "dht is not"),
    ("bwd", dict(dh0=Y + 4), "dh0 is not"),
])
def test_lin_output_refusals(which, kw, text):
    refused(B.GDR_EINVAL, text, lin_call, which, lin(), **kw)


@pytest.mark.parametrize("shape,kw,text", [
    (dict(T=2), {}, "T == 1"),
    (dict(T=1, cu_seqlens=[0, 1]), {}, "T == 1"),
    (dict(T=1), dict(h0=H0), "not from h0"),
    (dict(T=1), dict(q=None), "input q"),
    (dict(T=1), dict(o=None), "o is NULL"),
    (dict(T=1), dict(o=Y + 8), "o is not"),
    (dict(T=1), dict(state=None), "state is NULL"),
    (dict(T=1), dict(state=0xc00004), "state is not 16-byte"),
    (dict(T=1), dict(P=-1), "P (-1)"),
    (dict(T=1, B=5, N=5), dict(P=4), "as many states"),
    (dict(T=1), dict(slots=0xd00002), "slots is not 4-byte"),
])
def test_lin_step_refusals(shape, kw, text):
    refused(B.GDR_EINVAL, text, lin_call, "step", lin(**shape), **kw)


def test_a_forward_workspace_is_too_small_for_a_backward():
    p = lin(T=30000, H=4, Hk=2)
    n = B.gdr_lin_workspace_bytes(p)
    assert n < B.gdr_lin_workspace_bytes(p, True)
    refused(B.GDR_EWORKSPACE, f"workspace {n} bytes", lin_call, "bwd", p, ws_bytes=n)


def test_lin_workspace():
    states = 4 * 64 * 64
    one, two = (B.gdr_lin_workspace_bytes(lin(T=30000), b) for b in (False, True))
    assert two == 2 * one and one % (2 * states) == 0                    # a state for each segment, gradients alike
    assert B.gdr_lin_workspace_bytes(lin(T=64)) == 0                       # one segment: nothing between
    assert 0 < B.gdr_lin_workspace_bytes(lin(T=64, N=2, cu_seqlens=[0, 20, 64])) < states   # its table alone
    grouped = B.gdr_lin_workspace_bytes(lin(T=64, Hk=1), True)
    assert grouped == 64 * 2 * 64 * 4                                    # dq or dk for each value head


# ---- quantisation ----

def quant_call(prob, x=X, q=Y, scales=H0, null=False):
    call("gdr_quant", None if null else prob.ref, x, q, scales, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=3), B.GDR_EINVAL, "dtype"),
    (dict(rows=-1), B.GDR_EINVAL, "bad rows/cols"),
    (dict(cols=-1), B.GDR_EINVAL, "bad rows/cols"),
    (dict(block=64), B.GDR_EUNSUPPORTED, "block 64"),
    (dict(block=0), B.GDR_EUNSUPPORTED, "block 0"),
    (dict(block=-128), B.GDR_EUNSUPPORTED, "block -128"),
    (dict(transpose=2), B.GDR_EINVAL, "transpose 2"),
    (dict(rows=1 << 31, cols=1), B.GDR_EUNSUPPORTED, "too large"),
    (dict(rows=1, cols=1 << 31), B.GDR_EUNSUPPORTED, "too large"),
    (dict(rows=128 << 12, cols=128 << 12), B.GDR_EUNSUPPORTED, "too large"),     # 2^24 tiles
    (dict(rows=(1 << 63) - 1, cols=(1 << 63) - 1), B.GDR_EUNSUPPORTED, "too large"),
])
def test_quant_shape_validation(kw, status, text):
    refused(status, text, quant_call, B.QuantProblem(**{**dict(rows=4, cols=128, dtype=0), **kw}))


@pytest.mark.parametrize("kw,text", [
    (dict(null=True), "shape is NULL"),
    (dict(x=None), "x is NULL"),
    (dict(q=None), "q is NULL"),
    (dict(scales=None), "scales is NULL"),
    (dict(x=X + 8), "x is not 16-byte"),
    (dict(q=Y + 1), "q is not 16-byte"),
    (dict(scales=H0 + 4), "scales is not 16-byte"),
])
def test_quant_refusals(kw, text):
    refused(B.GDR_EINVAL, text, quant_call, B.QuantProblem(4, 128, B.GDR_BF16), **kw)


def test_quant_shapes():
    p = B.QuantProblem(300, 200, B.GDR_F32, block=128, transpose=True)
    assert p.q_shape == (200, 300) and p.scales_shape == (2, 3)
    p = B.QuantProblem(300, 200, B.GDR_F32)
    assert p.q_shape == (300, 200) and p.scales_shape == (300, 2)


# ---- product ----

def gemm_call(prob, a=X, sa=L, b=H0, sb=L, c=Y, ws=None, ws_bytes=0, null=False):
    call("gdr_gemm", None if null else prob.ref, a, sa, b, sb, ws, ws_bytes, c, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=2), B.GDR_EINVAL, "dtype"),
    (dict(M=-1), B.GDR_EINVAL, "bad M/N/K"),
    (dict(N=-1), B.GDR_EINVAL, "bad M/N/K"),
    (dict(K=0), B.GDR_EINVAL, "bad M/N/K"),
    (dict(block=64), B.GDR_EUNSUPPORTED, "block 64"),
    (dict(block=0), B.GDR_EUNSUPPORTED, "block 0"),
    (dict(M=(1 << 30) + 1, N=1), B.GDR_EUNSUPPORTED, "too large"),
    (dict(M=1, N=(1 << 30) + 1), B.GDR_EUNSUPPORTED, "too large"),
    (dict(K=(1 << 30) + 1), B.GDR_EUNSUPPORTED, "too large"),
    (dict(M=1 << 26, N=1), B.GDR_EUNSUPPORTED, "too large"),                  # 2^19 tiles
    (dict(M=1, N=1 << 26), B.GDR_EUNSUPPORTED, "too large"),
    (dict(M=1 << 30, N=1 << 30), B.GDR_EUNSUPPORTED, "too large"),
])
def test_gemm_shape_validation(kw, status, text):
    p = B.GemmProblem(**{**dict(M=64, N=128, K=256, dtype=0), **kw})
    refused(status, text, B.gdr_gemm_workspace_bytes, p)
    refused(status, text, gemm_call, p)


@pytest.mark.parametrize("M,N,K", [((1 << 26) - 128, 128, 1), (32, (1 << 26) - 128, 1 << 30), (33, (1 << 26) - 128, 1 << 30),
                                   (0, 1 << 30, 1 << 30), (1 << 30, 0, 1)])
def test_the_largest_products(M, N, K):
    for dtype in (B.GDR_BF16, B.GDR_F32):
        assert B.gdr_gemm_workspace_bytes(B.GemmProblem(M, N, K, dtype)) >= 0


@pytest.mark.parametrize("kw,status,text", [
    (dict(null=True), B.GDR_EINVAL, "shape is NULL"),
    (dict(a=None), B.GDR_EINVAL, "a is NULL"),
    (dict(sa=None), B.GDR_EINVAL, "a_scales is NULL"),
    (dict(b=None), B.GDR_EINVAL, "b is NULL"),
    (dict(sb=None), B.GDR_EINVAL, "b_scales is NULL"),
    (dict(c=None), B.GDR_EINVAL, "c is NULL"),
    (dict(a=X + 8), B.GDR_EINVAL, "a is not 16-byte"),
    (dict(sa=L + 4), B.GDR_EINVAL, "a_scales is not 16-byte"),
    (dict(b=H0 + 1), B.GDR_EINVAL, "b is not 16-byte"),
    (dict(sb=L + 8), B.GDR_EINVAL, "b_scales is not 16-byte"),
    (dict(c=Y + 2), B.GDR_EINVAL, "c is not 16-byte"),
])
def test_gemm_refusals(kw, status, text):
    refused(status, text, gemm_call, B.GemmProblem(64, 128, 256, B.GDR_BF16), **kw)


def test_gemm_workspace():
    split = B.GemmProblem(64, 512, 4096, B.GDR_BF16)
    n = B.gdr_gemm_workspace_bytes(split)
    assert n and n % (64 * 512 * 4) == 0                               # a sum for each run
    assert B.alloc_gemm_workspace(split, "cpu").numel() == n
    assert B.alloc_gemm_workspace(B.GemmProblem(64, 512, 128, B.GDR_BF16), "cpu") is None
    refused(B.GDR_EWORKSPACE, "workspace 0 bytes", gemm_call, split)
    refused(B.GDR_EWORKSPACE, f"workspace {n - 1} bytes", gemm_call, split, ws=WS, ws_bytes=n - 1)
    refused(B.GDR_EINVAL, "workspace is NULL", gemm_call, split, ws_bytes=n)
    refused(B.GDR_EINVAL, "256-byte aligned", gemm_call, split, ws=WS + 16, ws_bytes=n)


# ---- the binding's own checks (CPU tensors: a call that passed the others is refused for
# its device, so nothing here reaches the library) ----

WIDE = 1 << 32


@pytest.mark.parametrize("make", [
    lambda: lin(T=WIDE + 1), lambda: lin(H=WIDE + 2), lambda: lin(N=WIDE + 1), lambda: lin(Hk=WIDE),
    lambda: B.GemmProblem(WIDE + 1, 1, 1, 0), lambda: B.GemmProblem(1, 1, WIDE + 1, 0), lambda: B.GemmProblem(1, 1, 1, 0, WIDE + 128),
    lambda: B.QuantProblem(1 << 64, 1, 0), lambda: B.QuantProblem(1, 1, 0, WIDE + 1), lambda: B.QuantProblem(1, 1, WIDE),
])
def test_fields_beyond_the_abi_are_refused(make):
    refused(B.GDR_EUNSUPPORTED, "beyond", make)


def test_binding_checks_lin_tensors():
    p = lin(T=3, H=4, Hk=2)
    q, v = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(3, 4, 64, dtype=BF)
    t = {"q": q, "k": q, "v": v, "log_decay": torch.zeros(4), "h0": torch.zeros(1, 4, 64, 64)}
    ws, out = torch.zeros(256, dtype=torch.uint8), {"dq": q, "dk": q, "dv": v, "dh0": t["h0"]}
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_lin_fwd, p, t, ws, v)
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_lin_bwd, p, t, v, None, ws, out)
    refused(B.GDR_EINVAL, "q has 768", B.gdr_lin_fwd, p, {**t, "q": v}, ws, v)
    refused(B.GDR_EINVAL, "v has 384", B.gdr_lin_fwd, p, {**t, "v": q}, ws, v)
    refused(B.GDR_EINVAL, "k is torch.float32", B.gdr_lin_fwd, p, {**t, "k": q.float()}, ws, v)
    refused(B.GDR_EINVAL, "log_decay is torch.bfloat16", B.gdr_lin_fwd, p, {**t, "log_decay": torch.zeros(4, dtype=BF)}, ws, v)
    refused(B.GDR_EINVAL, "log_decay has 2", B.gdr_lin_fwd, p, {**t, "log_decay": torch.zeros(2)}, ws, v)
    refused(B.GDR_EINVAL, "h0 has 4096", B.gdr_lin_fwd, p, {**t, "h0": torch.zeros(64, 64)}, ws, v)
    refused(B.GDR_EINVAL, "ht is torch.bfloat16", B.gdr_lin_fwd, p, t, ws, v, ht=t["h0"].to(BF))
    refused(B.GDR_EINVAL, "k is not contiguous", B.gdr_lin_fwd, p, {**t, "k": torch.zeros(2, 3, 64, dtype=BF).transpose(0, 1)}, ws, v)
    refused(B.GDR_EINVAL, "dht has 2", B.gdr_lin_bwd, p, t, v, torch.zeros(2), ws, out)
    refused(B.GDR_EINVAL, "dk has 768", B.gdr_lin_bwd, p, t, v, None, ws, {**out, "dk": v})
    one = lin(T=1, B=3, N=3, H=4, Hk=2)
    st = torch.zeros(5, 4, 64, 64)
    refused(B.GDR_EINVAL, "state has shape", B.gdr_lin_step, one, {**t, "h0": None}, torch.zeros(5, 64), v)
    refused(B.GDR_EINVAL, "slots is torch.int64", B.gdr_lin_step, one, {**t, "h0": None}, st, v, slots=torch.zeros(3, dtype=torch.int64))
    refused(B.GDR_EINVAL, "slots has 2", B.gdr_lin_step, one, {**t, "h0": None}, st, v, slots=torch.zeros(2, dtype=torch.int32))
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_lin_step, one, {**t, "h0": None}, st, v)
    refused(B.GDR_EINVAL, "cu_seqlens has 2 entries", lin, N=2, cu_seqlens=[0, 300])


def test_binding_checks_projection_tensors():
    x, q, s = torch.zeros(3, 200, dtype=BF), torch.zeros(3, 200).to(E4), torch.zeros(3, 2)
    p = B.QuantProblem(3, 200, B.GDR_BF16)
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_quant, p, x, q, s)
    refused(B.GDR_EINVAL, "x is torch.float32", B.gdr_quant, p, x.float(), q, s)
    refused(B.GDR_EINVAL, "q is torch.uint8", B.gdr_quant, p, x, torch.zeros(3, 200, dtype=torch.uint8), s)
    refused(B.GDR_EINVAL, "scales has 3", B.gdr_quant, p, x, q, s[:, :1].contiguous())
    refused(B.GDR_EINVAL, "x is not contiguous", B.gdr_quant, p, torch.zeros(200, 3, dtype=BF).t(), q, s)
    g = B.GemmProblem(3, 5, 200, B.GDR_F32)
    b, sb, c = torch.zeros(5, 200).to(E4), torch.zeros(1, 2), torch.zeros(3, 5)
    refused(B.GDR_EINVAL, "expected a GPU", B.gdr_gemm, g, q, s, b, sb, c)
    refused(B.GDR_EINVAL, "a is torch.bfloat16", B.gdr_gemm, g, x, s, b, sb, c)
    refused(B.GDR_EINVAL, "b has 600", B.gdr_gemm, g, q, s, q, sb, c)
    refused(B.GDR_EINVAL, "a_scales has 2", B.gdr_gemm, g, q, sb, b, sb, c)
    refused(B.GDR_EINVAL, "b_scales has 6", B.gdr_gemm, g, q, s, b, s, c)
    refused(B.GDR_EINVAL, "c is torch.bfloat16", B.gdr_gemm, g, q, s, b, sb, c.to(BF))


class Stream:
    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 0


class Reached(Exception):
    pass


class Library:
    """Stands in for the loaded library: no call may get this far."""

    def __getattr__(self, name):
        def entry(*args):
            raise Reached(name)
        return entry


@pytest.mark.parametrize("name", ["gdr_lin_fwd", "gdr_lin_bwd", "gdr_lin_step", "gdr_quant", "gdr_gemm"])
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    """The tensors are on the current device, so the call has to run there."""
    x, ws, S = torch.zeros(2, 64, dtype=BF), torch.zeros(256, dtype=torch.uint8), torch.zeros(2, 1, 64, 64)
    t = {"q": x, "k": x, "v": x, "log_decay": torch.zeros(1)}
    p, one = lin(T=2, H=1), lin(B=2, N=2, T=1, H=1)
    q, s = x.to(E4), torch.zeros(2, 1)
    run = {
        "gdr_lin_fwd": lambda st: B.gdr_lin_fwd(p, t, ws, x, stream=st),
        "gdr_lin_bwd": lambda st: B.gdr_lin_bwd(p, t, x, None, ws, {"dq": x, "dk": x, "dv": x}, stream=st),
        "gdr_lin_step": lambda st: B.gdr_lin_step(one, t, S, x, stream=st),
        "gdr_quant": lambda st: B.gdr_quant(B.QuantProblem(2, 64, B.GDR_BF16), x, q, s, stream=st),
        "gdr_gemm": lambda st: B.gdr_gemm(B.GemmProblem(2, 2, 64, B.GDR_F32), q, s, q, s[:1], torch.zeros(2, 2), stream=st),
    }[name]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_check_tensors", lambda specs: None)     # they are on the CPU here
    monkeypatch.setattr(B, "load_library", lambda: Library())
    refused(B.GDR_EINVAL, "stream is on cuda:1", run, Stream(1))
    for same in (Stream(0), 0):
        with pytest.raises(Reached, match=name):
            run(same)
