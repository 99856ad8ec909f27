"""Refusals of the scored routing and the 8-bit float entry points, on the CPU: every
check runs before anything is enqueued (ctypes with addresses that are never read),
and the binding's own checks of tensors."""
import ctypes

import pytest

import quantized_moe_ffn_amd as qm

P = ctypes.c_void_p


def _r():
    return qm.moe_routing(*(P(8 * (i + 1)) for i in range(7)))


def _spec(**kw):
    d = dict(score=1, n_group=1, topk_group=1, group_top=1, renorm=1, scale=1.0, bias=None)
    d.update(kw)
    return qm.moe_route_spec(*(d[n] for n, _ in qm.moe_route_spec._fields_))


def _route(T=2, E=64, k=4, spec=None, logits=4096, ws=None, n=0, r=None):
    return qm.load_library().moe_route_scored(P(logits), T, E, k, ctypes.byref(spec or _spec()),
                                              ctypes.byref(r or _r()), P(ws), n, None)


@pytest.mark.parametrize("kw,st,msg", [
    (dict(T=0), 1, "T = 0"), (dict(E=0), 1, "E = 0"), (dict(E=1025), 1, "E = 1025"), (dict(k=0), 1, "k = 0"),
    (dict(k=17), 1, "k = 17"), (dict(E=3, k=4), 1, "k = 4"), (dict(T=1 << 27, k=16), 1, "too large"),
    (dict(logits=4097), 1, "4-byte aligned"), (dict(logits=0), 1, "logits is NULL"),
    (dict(spec=_spec(score=2)), 1, "spec.score = 2"), (dict(spec=_spec(n_group=0)), 1, "n_group = 0"),
    (dict(spec=_spec(n_group=3)), 1, "n_group = 3"), (dict(E=256, spec=_spec(n_group=128)), 1, "n_group = 128"),
    (dict(spec=_spec(n_group=8, topk_group=0)), 1, "topk_group = 0"), (dict(spec=_spec(n_group=8, topk_group=9)), 1, "topk_group = 9"),
    (dict(k=9, spec=_spec(n_group=8, topk_group=1)), 1, "hold fewer"), (dict(spec=_spec(group_top=3)), 1, "group_top = 3"),
    (dict(spec=_spec(n_group=64, topk_group=8, group_top=2)), 1, "group_top = 2"),
    (dict(spec=_spec(scale=float("nan"))), 1, "scale must be finite"), (dict(spec=_spec(scale=float("inf"))), 1, "scale"),
    (dict(spec=_spec(bias=4098)), 1, "bias"), (dict(T=100), 3, "routing workspace"),
    (dict(T=100, ws=4096, n=8), 3, "routing workspace"), (dict(T=100, ws=4098, n=1 << 30), 1, "4-byte aligned"),
    (dict(r=qm.moe_routing()), 1, "moe_routing"),
])
def test_route_scored_refusals(kw, st, msg):
    assert _route(**kw) == st, qm.moe_last_error()
    assert msg in qm.moe_last_error()


def test_route_scored_needs_a_spec():
    assert qm.load_library().moe_route_scored(P(4096), 1, 8, 2, None, ctypes.byref(_r()), None, 0, None) == 1
    assert "spec is NULL" in qm.moe_last_error()


def _quant(x=4096, xt=30, ldx=256, T=2, H=256, xq=4096, xs=4096):
    return qm.load_library().moe_quantize_fp8(P(x), xt, ldx, T, H, P(xq), P(xs), None)


@pytest.mark.parametrize("kw,st,msg", [
    (dict(x=0), 1, "NULL"), (dict(xq=0), 1, "NULL"), (dict(xs=0), 1, "NULL"), (dict(xt=2), 2, "x_type = 2"),
    (dict(T=0), 1, "T = 0"), (dict(H=0), 1, "H = 0"), (dict(H=24, ldx=24), 1, "H = 24"), (dict(ldx=128), 1, "ldx = 128"),
    (dict(ldx=260), 1, "16-byte aligned"), (dict(xt=0, ldx=258), 1, "16-byte aligned"), (dict(x=4104), 1, "16-byte aligned"),
    (dict(xq=4100), 1, "xq 8-byte"), (dict(xs=4098), 1, "xs 4-byte"),
])
def test_quantize_refusals(kw, st, msg):
    assert _quant(**kw) == st, qm.moe_last_error()
    assert msg in qm.moe_last_error()


def _mat(rows=256, cols=512, data=4096, scale=4096, row_stride=None, expert_stride=None):
    rs = cols if row_stride is None else row_stride
    return qm.moe_fp8_matrix(data, scale, rows, cols, rs, rows * rs if expert_stride is None else expert_stride)


def _mm(w=None, xq=4096, xs=4096, T=2, y=4096, yt=30, ldy=256):
    return qm.load_library().moe_matmul_fp8(P(xq), P(xs), T, ctypes.byref(w or _mat()), P(y), yt, ldy, None)


@pytest.mark.parametrize("kw,st,msg", [
    (dict(xq=0), 1, "NULL"), (dict(y=0), 1, "NULL"), (dict(xs=0), 1, "NULL"), (dict(T=0), 1, "T = 0"), (dict(yt=8), 2, "y_type = 8"),
    (dict(w=_mat(data=0)), 1, "data or scale is NULL"), (dict(w=_mat(scale=0)), 1, "data or scale is NULL"),
    (dict(w=_mat(rows=0)), 1, "0 x 512"), (dict(w=_mat(cols=8)), 1, "256 x 8"), (dict(w=_mat(cols=520)), 1, "multiple of 16"),
    (dict(w=_mat(row_stride=496)), 1, "row_stride = 496"), (dict(w=_mat(row_stride=520)), 1, "row_stride = 520"),
    (dict(w=_mat(row_stride=(1 << 23) + 16)), 1, "too large"), (dict(w=_mat(expert_stride=8)), 1, "expert_stride = 8"),
    (dict(w=_mat(data=4104)), 1, "16-byte aligned"), (dict(ldy=255), 1, "ldy = 255"), (dict(xq=4104), 1, "xq must be 16-byte"),
    (dict(y=4097), 1, "element aligned"), (dict(y=4098, yt=0), 1, "element aligned"),
])
def test_matmul_refusals(kw, st, msg):
    assert _mm(**kw) == st, qm.moe_last_error()
    assert msg in qm.moe_last_error()


def _layer(E=8, H=256, I=128, shared=False, **over):
    L = qm.moe_fp8_layer()
    L.n_experts, L.hidden, L.inter, L.has_shared = E, H, I, int(shared)
    L.gate, L.up, L.down = _mat(I, H), _mat(I, H), _mat(H, I)
    if shared:
        L.sh_gate, L.sh_up, L.sh_down = _mat(I, H), _mat(I, H), _mat(H, I)
    for n, v in over.items():
        setattr(L, n, v)
    return L


def _fwd(L=None, T=2, k=2, x=4096, xt=30, flags=0, out=4096, scale=None, ws=4096, n=1 << 40, spec=None, logits=4096, r=None):
    lib = qm.load_library()
    return lib.moe_forward_fp8(ctypes.byref(L or _layer()), ctypes.byref(spec or _spec()), P(logits), P(x), xt, T, k, flags,
                               ctypes.byref(r or _r()), P(scale), P(out), P(ws), n, None)


@pytest.mark.parametrize("kw,st,msg", [
    (dict(L=_layer(E=0)), 1, "n_experts = 0"), (dict(L=_layer(H=192)), 1, "hidden = 192"), (dict(L=_layer(I=64)), 1, "inter = 64"),
    (dict(L=_layer(H=16512)), 2, "16512"), (dict(T=0), 1, "T = 0"), (dict(k=9), 1, "k = 9"), (dict(T=1 << 24), 1, "hidden = 4294967296"),
    (dict(L=_layer(up=_mat(128, 512))), 1, "up is 128 x 512"), (dict(L=_layer(down=_mat(256, 128, expert_stride=256 * 127))), 1, "down.expert_stride"),
    (dict(L=_layer(shared=True, sh_down=qm.moe_fp8_matrix())), 1, "sh_down"), (dict(x=0), 1, "x or out is NULL"),
    (dict(out=0), 1, "x or out is NULL"), (dict(xt=12), 2, "x_type = 12"), (dict(flags=1), 1, "ffn_flags = 0x1"),
    (dict(scale=4096), 1, "without a shared expert"), (dict(x=4104), 1, "16-byte aligned"), (dict(out=4104), 1, "16-byte aligned"),
    (dict(L=_layer(shared=True), scale=4097), 1, "4-byte aligned"), (dict(ws=0), 3, "fp8 forward workspace"),
    (dict(n=100), 3, "fp8 forward workspace"), (dict(ws=4096 + 128), 1, "256-byte aligned"), (dict(logits=0), 1, "logits is NULL"),
    (dict(spec=_spec(n_group=3)), 1, "n_group = 3"), (dict(r=qm.moe_routing()), 1, "moe_routing"),
])
def test_forward_refusals(kw, st, msg):
    assert _fwd(**kw) == st, qm.moe_last_error()
    assert msg in qm.moe_last_error()


@pytest.mark.parametrize("kw,st,msg", [
    (dict(xq=0), 1, "NULL"), (dict(yp=0), 1, "NULL"), (dict(L=_layer(shared=True)), 1, "y_shared is NULL"), (dict(xq=4104), 1, "16-byte"),
    (dict(yp=4100), 1, "16-byte"), (dict(n=64), 3, "fp8 FFN workspace"), (dict(ws=4100), 1, "256-byte aligned"), (dict(T=0), 1, "T = 0"),
])
def test_expert_ffn_refusals(kw, st, msg):
    a = dict(L=_layer(), xq=4096, xs=4096, yp=4096, ys=None, ws=4096, n=1 << 40, T=2)
    a.update(kw)
    got = qm.load_library().moe_expert_ffn_fp8(ctypes.byref(a["L"]), ctypes.byref(_r()), a["T"], 2, P(a["xq"]), P(a["xs"]),
                                               P(a["yp"]), P(a["ys"]), P(a["ws"]), a["n"], None)
    assert got == st, qm.moe_last_error()
    assert msg in qm.moe_last_error()


def test_workspaces_grow_with_the_work():
    lib = qm.load_library()
    for shared in (False, True):
        L = _layer(E=64, H=1024, I=256, shared=shared)
        last = 0
        for T in (1, 2, 31, 33, 100, 5000, 100000):
            f = lib.moe_ffn_fp8_workspace_bytes(ctypes.byref(L), T, 4)
            rows = T * 4 + (T if shared else 0)
            assert f >= rows * 256 + rows * 2 * 4 and f >= last
            last = f
            a, b = (lib.moe_forward_fp8_workspace_bytes(ctypes.byref(L), T, 4, fl) for fl in (0, 16))
            assert a >= b >= f + T * 1024
            if T * 4 > 64:   # the per-pair outputs pass through the workspace
                assert a > b >= f + T * 1024 + rows * 1024 * 2
    assert lib.moe_forward_fp8_workspace_bytes(ctypes.byref(L), 1, 4, 2) == 0
    assert lib.moe_forward_fp8_workspace_bytes(None, 1, 4, 0) == 0 and lib.moe_ffn_fp8_workspace_bytes(ctypes.byref(L), 0, 4) == 0


def test_binding_checks_tensors_before_the_call():
    torch = pytest.importorskip("torch")
    f8 = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    w = qm.Fp8Matrix(torch.zeros(1, 256, 256, dtype=torch.uint8), torch.zeros(1, 2, 2))
    x, d, y = torch.zeros(4, 256), torch.zeros(4, 2), torch.zeros(4, 256)
    for bad, msg in [
        (lambda: qm.Fp8Matrix(torch.zeros(1, 8, 16), torch.zeros(1, 1, 1)), "e4m3 codes"),
        (lambda: qm.Fp8Matrix(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(1, 1, 1)), "rows"),
        (lambda: qm.Fp8Matrix(torch.zeros(1, 8, 16, dtype=torch.uint8), torch.zeros(1, 1, 2)), "scale: "),
        (lambda: qm.Fp8Matrix(torch.zeros(1, 16, 8, dtype=torch.uint8).transpose(1, 2), torch.zeros(1, 1, 1)), "columns"),
        (lambda: qm.moe_quantize_fp8(x, f8[:3], d), "xq: "),
        (lambda: qm.moe_quantize_fp8(x, x, d), "e4m3 codes"),
        (lambda: qm.moe_quantize_fp8(x.t(), f8.t(), d), "columns"),
        (lambda: qm.moe_quantize_fp8(x, f8, d.int()), "xs: "),
        (lambda: qm.moe_quantize_fp8(x.double(), f8, d), "dtype"),
        (lambda: qm.moe_quantize_fp8(x, f8, d), "on a GPU"),
        (lambda: qm.moe_matmul_fp8(f8[:, :128].contiguous(), d, w, y), "xq: "),
        (lambda: qm.moe_matmul_fp8(f8, d[:, :1], w, y), "xs: "),
        (lambda: qm.moe_matmul_fp8(f8, d, w, y[:, :255]), "y has shape"),
        (lambda: qm.moe_matmul_fp8(f8, d, w, y.t().contiguous().t()), "contiguous columns"),
        (lambda: qm.moe_matmul_fp8(f8, d, w, y.int()), "dtype"),
        (lambda: qm.RouteSpec("relu"), "score"),
        (lambda: qm.RouteSpec(bias=torch.zeros(8, dtype=torch.float64)), "bias: "),
        (lambda: qm.Fp8Layer(w, w, w, (w, w)), "shared"),
    ]:
        with pytest.raises(ValueError, match=msg):
            bad()
    r = qm.Routing(4, 8, 2, "cpu")
    lg = torch.zeros(4, 8)
    for bad, msg in [
        (lambda: qm.moe_route_scored(lg, 3, r, qm.RouteSpec()), "routing buffers"),
        (lambda: qm.moe_route_scored(lg.half(), 2, r, qm.RouteSpec()), "logits: "),
        (lambda: qm.moe_route_scored(lg, 2, r, qm.RouteSpec(bias=torch.zeros(7))), "bias has 7"),
        (lambda: qm.moe_route_scored(lg, 2, r, qm.RouteSpec()), "on a GPU"),
    ]:
        with pytest.raises(ValueError, match=msg):
            bad()
