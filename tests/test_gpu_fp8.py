"""The 8-bit float quantiser, product and expert layer against the 64-bit reference."""
import numpy as np
import pytest

from tests import fp8_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _qm():
    import quantized_moe_ffn_amd as m
    m.load_library()
    return m


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _quantize(m, x):
    T, H = x.shape
    q = torch.full((T, H), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    d = torch.full((T, ref.nb(H)), float("nan"), device=DEV)
    m.moe_quantize_fp8(x, q, d)
    return q, d


def _weights(g, E, N, K):
    """Random finite codes and scales, on the host and on the device."""
    q = g.integers(0, 256, (E, N, K), dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] ^= 1
    s = (g.uniform(0.2, 1.0, (E, ref.nb(N), ref.nb(K))) / (100 * np.sqrt(K))).astype(np.float32)
    return q, s


def _matrix(m, q, s):
    return m.Fp8Matrix(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV))


# ------------------------------------------------------------------ quantiser


@pytest.mark.parametrize("xt", sorted(DT))
@pytest.mark.parametrize("T,H", [(1, 16), (1, 2048), (3, 2560), (5, 144), (37, 128), (33, 1008), (300, 256)])
def test_quantize(xt, T, H):
    m = _qm()
    print("quantize", xt, T, H, flush=True)
    g = np.random.default_rng(T * 1000 + H)
    x = torch.from_numpy(g.standard_normal((T, H)) * np.exp(g.standard_normal((T, 1)) * 3)).clamp(-6e4, 6e4).to(DT[xt])
    x[T // 2, : min(H, 128)] = 0
    q, d = _quantize(m, x.to(DEV))
    m.moe_check_device_errors()
    x64 = x.double().numpy()
    rq, rd = ref.quantize(x64)
    assert np.array_equal(d.cpu().numpy(), rd.astype(np.float32))
    got = _codes(q)
    if xt == "f32":   # x * 448 / a carries fp32 roundings: a code may differ where the exact quotient is that near a tie
        a = np.repeat(rd * 448, 128, 1)[:, :H]
        quot = x64 * 448 / np.where(a > 0, a, 1)
        hit, _ = ref.near_midpoint(quot, np.abs(quot) * 4 * ref.U)
        assert (np.array_equal(got[~hit], rq[~hit])) and hit.mean() < 1e-3
    else:
        assert np.array_equal(got & 0x7F, rq & 0x7F)
        nz = (rq & 0x7F) != 0
        assert np.array_equal(got[nz], rq[nz])


@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_quantize_ties_are_those_of_exact_arithmetic(xt):
    """Rows whose maximum is a multiple of 7 put 448/a times a short input exactly between two codes."""
    m = _qm()
    rows = []
    for a in (7, 14, 21, 28, 35, 49, 56, 63, 77, 91, 105, 112, 119):
        v = np.arange(-a, a + 1, dtype=np.float64)
        rows.append(np.pad(v, (0, 256 - len(v)))[:256])
    x = torch.tensor(np.array(rows)).to(DT[xt])
    q, d = _quantize(m, x.to(DEV))
    rq, rd = ref.quantize(x.double().numpy())
    assert np.array_equal(ref.decode(_codes(q)), ref.decode(rq)) and np.array_equal(d.cpu().numpy(), rd.astype(np.float32))


def test_quantize_range_limits():
    m = _qm()
    x = np.zeros((6, 128), np.float32)
    x[0, :3] = [3.4028235e38, -3.4028235e38, 1e38]
    x[1, :3] = [1e-45, -1e-44, 1e-40]
    x[2, :3] = [2.0 ** -116, 2.0 ** -117, -2.0 ** -126]
    x[3, :2] = [1.0, 2.0 ** -17]
    x[4, :3] = [448.0, 2.0 ** -9, 2.0 ** -10]
    q, d = _quantize(m, torch.from_numpy(x).to(DEV))
    m.moe_check_device_errors()
    rq, rd = ref.quantize(x.astype(np.float64))
    assert np.array_equal(ref.decode(_codes(q)), ref.decode(rq)) and np.array_equal(d.cpu().numpy(), rd.astype(np.float32))
    assert np.isfinite(d.cpu().numpy()).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_non_finite_blocks_are_zero_and_raise(bad):
    m = _qm()
    x = torch.randn(4, 512, device=DEV, dtype=torch.bfloat16)
    ok_q, ok_d = _quantize(m, x)
    y = x.clone()
    y[2, 300] = bad
    q, d = _quantize(m, y)
    with pytest.raises(m.MoeError, match="non-finite activation"):
        m.moe_check_device_errors()
    assert not _codes(q)[2, 256:384].any() and d[2, 2] == 0
    keep = torch.ones(4, 512, dtype=torch.bool)
    keep[2, 256:384] = False
    assert np.array_equal(_codes(q)[keep.numpy()], _codes(ok_q)[keep.numpy()])


def test_quantize_strided_rows_and_untouched_neighbours():
    m = _qm()
    big = torch.randn(9, 400, device=DEV, dtype=torch.float16)
    x = big[:, 8:8 + 272]
    q = torch.full((10, 272), 0x11, dtype=torch.uint8, device=DEV)
    d = torch.full((10, 3), -1.0, device=DEV)
    m.moe_quantize_fp8(x, q[:9], d[:9])
    rq, rd = ref.quantize(x.double().cpu().numpy())
    assert np.array_equal(ref.decode(q[:9].cpu().numpy()), ref.decode(rq))
    assert (q[9] == 0x11).all() and (d[9] == -1).all()


# ------------------------------------------------------------------ product


def _matmul_case(m, T, N, K, yt, seed, ldy=None):
    g = np.random.default_rng(seed)
    x = torch.from_numpy((g.standard_normal((T, K)) * np.exp(g.standard_normal((T, 1)))).astype(np.float32)).to(DEV)
    q, d = _quantize(m, x)
    wq, ws = _weights(g, 1, N, K)
    big = torch.full((T + 1, ldy or N), -7.0, dtype=DT[yt], device=DEV)
    y = big[:T, :N]
    m.moe_matmul_fp8(q, d, _matrix(m, wq, ws), y)
    m.moe_check_device_errors()
    r, bound = ref.matmul(_codes(q), d.cpu().numpy(), wq[0], ws[0], fast=yt != "f32")
    half = 0 if yt == "f32" else torch.finfo(DT[yt]).eps / 2
    tiny = 2.0 ** -25 if yt == "f16" else 0
    got = y.double().cpu().numpy()
    assert (np.abs(got - r) <= bound * (1 + half) + np.abs(r) * half + tiny).all(), np.abs(got - r).max()
    assert (big[T] == -7).all() and (big[:, N:] == -7).all()


@pytest.mark.parametrize("yt", sorted(DT))
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 2048, 2560), (1, 130, 48), (2, 1000, 2000), (7, 17, 128), (16, 256, 512),
                                   (17, 300, 1024), (33, 129, 272), (64, 64, 4096), (65, 515, 640), (130, 256, 144),
                                   (333, 1000, 2000), (520, 700, 1168)])
def test_matmul(T, N, K, yt):
    m = _qm()
    print("matmul", T, N, K, yt, flush=True)
    _matmul_case(m, T, N, K, yt, T * 31 + N + K)


@pytest.mark.parametrize("T", [1, 5, 40, 200, 600])
@pytest.mark.parametrize("ldy", [301, 320])
def test_matmul_output_rows_at_any_distance(T, ldy):
    m = _qm()
    _matmul_case(m, T, 299, 384, "bf16", T, ldy)


def test_matmul_deep_sum():
    m = _qm()
    _matmul_case(m, 3, 40, 16384, "f32", 1)
    _matmul_case(m, 70, 40, 16384, "f32", 2)


@pytest.mark.parametrize("T", [1, 20, 100, 700])
def test_matmul_integers_are_exact(T):
    """Small integers and power-of-two scales: every sum is an fp32 integer."""
    m = _qm()
    g = np.random.default_rng(T)
    N, K = 272, 656
    xv, wv = g.integers(-3, 4, (T, K)).astype(np.float64), g.integers(-3, 4, (N, K)).astype(np.float64)
    xs = 2.0 ** g.integers(-2, 3, (T, ref.nb(K))).astype(np.float32)
    ws = 2.0 ** g.integers(-2, 3, (ref.nb(N), ref.nb(K))).astype(np.float32)
    y = torch.empty(T, N, device=DEV)
    m.moe_matmul_fp8(torch.from_numpy(ref.encode(xv)).to(DEV), torch.from_numpy(xs).to(DEV),
                     _matrix(m, ref.encode(wv)[None], ws[None]), y)
    r, _ = ref.matmul(ref.encode(xv), xs, ref.encode(wv), ws)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), r)


@pytest.mark.parametrize("yt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,N,K,odd_xs", [(2100, 2060, 512, False),     # tiles of 256 x 128
                                          (2100, 2060, 640, False), (2100, 2060, 512, True),   # the same without groups of four blocks
                                          (2900, 2900, 1024, False),    # 256 x 256 for 16-bit outputs
                                          (2900, 2900, 640, False), (20, 12300, 512, False),
                                          (1050, 8192 - 3, 8704, False)])   # more than 64 blocks
def test_matmul_many_rows(T, N, K, odd_xs, yt):
    """Large tiles: small integers, whose sums are exact, in all places; drawn values against 64 bits at sampled rows."""
    m = _qm()
    print("matmul", T, N, K, odd_xs, yt, flush=True)
    g = np.random.default_rng(T + N + K)
    xv, wv = (torch.from_numpy(g.integers(-1, 2, n).astype(np.float32)).to(DEV) for n in ((T, K), (N, K)))
    xs = torch.empty(T * ref.nb(K) + 1, device=DEV)[int(odd_xs):][:T * ref.nb(K)].view(T, ref.nb(K)).fill_(1.0)
    ws = np.full((1, ref.nb(N), ref.nb(K)), 0.5, np.float32)
    big = torch.full((T + 1, N + 5), -7.0, dtype=DT[yt], device=DEV)
    table = torch.from_numpy(ref.encode(np.array([-1.0, 0.0, 1.0]))).to(DEV)
    def codes(v):
        return table[(v + 1).long()]
    m.moe_matmul_fp8(codes(xv), xs, m.Fp8Matrix(codes(wv)[None], torch.from_numpy(ws).to(DEV)), big[:T, :N])
    want = (xv @ wv.T) * 0.5    # fp32 holds every partial sum
    assert torch.equal(big[:T, :N], want.to(DT[yt]))
    assert (big[T] == -7).all() and (big[:, N:] == -7).all()
    q, d = _quantize(m, torch.from_numpy(g.standard_normal((T, K)).astype(np.float32)).to(DEV))
    xs.copy_(d)
    wq, s = _weights(g, 1, N, K)
    y = torch.empty(T, N, dtype=DT[yt], device=DEV)
    m.moe_matmul_fp8(q, xs, _matrix(m, wq, s), y)
    m.moe_check_device_errors()
    at = np.unique(np.concatenate([[0, T - 1], g.integers(0, T, 30)]))
    r, bound = ref.matmul(_codes(q)[at], d.cpu().numpy()[at], wq[0], s[0], fast=yt != "f32")
    half = 0 if yt == "f32" else torch.finfo(DT[yt]).eps / 2
    got = y.double().cpu().numpy()[at]
    assert (np.abs(got - r) <= bound * (1 + half) + np.abs(r) * half + (2.0 ** -25 if yt == "f16" else 0)).all()


def test_matmul_strided_weights():
    m = _qm()
    g = np.random.default_rng(4)
    q, s = _weights(g, 1, 200, 1024)
    big = torch.from_numpy(q).to(DEV)
    view = big[:, 3:150, 256:768]          # rows at a distance of 1,024 bytes, columns of two blocks on
    sc = torch.from_numpy(g.uniform(0.5, 1, (1, 2, 4)).astype(np.float32)).to(DEV)
    x, d = _quantize(m, torch.randn(9, 512, device=DEV))
    y = torch.empty(9, 147, device=DEV)
    m.moe_matmul_fp8(x, d, m.Fp8Matrix(view, sc), y)
    r, bound = ref.matmul(_codes(x), d.cpu().numpy(), view[0].cpu().numpy(), sc[0].cpu().numpy())
    assert (np.abs(y.cpu().numpy() - r) <= bound).all()


def test_matmul_nan_codes_reach_their_outputs_only():
    m = _qm()
    g = np.random.default_rng(6)
    for T in (2, 40, 200):
        q, s = _weights(g, 1, 140, 400)
        q[0, 77, 395] = 0x7F
        x, d = _quantize(m, torch.rand(T, 400, device=DEV) + 0.5)
        y = torch.empty(T, 140, device=DEV)
        m.moe_matmul_fp8(x, d, _matrix(m, q, s), y)
        bad = torch.isnan(y).cpu().numpy()
        assert bad[:, 77].all() and bad.sum() == T


# ------------------------------------------------------------------ expert layer


def _layer(m, g, E, H, I, shared):
    host = {n: _weights(g, E, *rc) for n, rc in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))}
    if shared:
        host.update({"sh_" + n: _weights(g, 1, *rc) for n, rc in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))})
    mats = {n: _matrix(m, *v) for n, v in host.items()}
    sh = tuple(mats["sh_" + n] for n in ("gate", "up", "down")) if shared else None
    return m.Fp8Layer(mats["gate"], mats["up"], mats["down"], sh), host


def _reference(host, xq, xs, idx, fast=False):
    """y_pair and y_shared with their bounds."""
    T, k = idx.shape
    H = xq.shape[1]
    y, dy = np.zeros((T * k, H)), np.zeros((T * k, H))
    for e in np.unique(idx):
        p = np.nonzero(idx.reshape(-1) == e)[0]
        y[p], dy[p] = ref.expert(xq[p // k], xs[p // k], *((host[n][0][e], host[n][1][e]) for n in ("gate", "up", "down")), fast=fast)
    if "sh_gate" not in host:
        return y, dy, None, None
    return (y, dy) + ref.expert(xq, xs, *((host["sh_" + n][0][0], host["sh_" + n][1][0]) for n in ("gate", "up", "down")), fast=fast)


def _expected(host, xq, xs, idx, w, sc, xt, flags):
    """The layer's output rows for the given tokens, and the limit of their error."""
    T, k = idx.shape
    H = xq.shape[1]
    y, dy, sh, dsh = _reference(host, xq, xs, idx, fast=xt == "bf16")
    def handed(v, dv):   # the 16-bit hand-off: fp16 times a power of two below twice the block's largest
        if not flags:
            return dv
        big = np.repeat((np.abs(v) + dv).reshape(len(v), -1, 64).max(axis=2), 64, 1)
        return dv + 2.0 ** -11 * (np.abs(v) + dv) + 2.0 ** -25 * big
    dy = handed(y, dy)
    a = np.abs(w)[:, :, None]
    o = (w[:, :, None] * y.reshape(T, k, H)).sum(1)
    mag = (a * np.abs(y).reshape(T, k, H)).sum(1)
    do = (a * dy.reshape(T, k, H)).sum(1)
    if sh is not None:
        s = sc.double().cpu().numpy()[:, None]
        o = o + s * sh
        do += s * handed(sh, dsh)
        mag += s * np.abs(sh)
    do += (k + 3) * ref.U * (mag + do)                             # fp32 weights, k + 1 fmas
    half = 0 if xt == "f32" else torch.finfo(DT[xt]).eps / 2
    return o, do * (1 + half) + np.abs(o) * half + (2.0 ** -25 if xt == "f16" else 0)


LAYERS = [  # T, E, k, H, I, shared
    (1, 8, 2, 256, 256, False), (1, 40, 3, 1024, 384, True), (1, 256, 8, 2048, 512, False), (3, 16, 10, 640, 128, True),
    (4, 8, 2, 256, 256, False), (9, 6, 4, 384, 256, True), (30, 5, 1, 128, 128, False), (61, 12, 4, 512, 256, False),
    (100, 4, 2, 256, 384, True), (300, 3, 3, 384, 128, False), (700, 8, 2, 256, 256, True),
]


@pytest.mark.parametrize("T,E,k,H,I,shared", LAYERS)
def test_expert_ffn(T, E, k, H, I, shared):
    m = _qm()
    print("ffn", T, E, k, H, I, shared, flush=True)
    g = np.random.default_rng(T + E + H)
    L, host = _layer(m, g, E, H, I, shared)
    lg = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).to(DEV)
    r = m.Routing(T, E, k, DEV)
    m.moe_route_scored(lg, k, r, m.RouteSpec(), torch.empty(max(4, m.moe_route_workspace_bytes(T, E, k)), dtype=torch.uint8, device=DEV))
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(DEV)
    q, d = _quantize(m, x)
    yp = torch.full((T * k + 1, H), -3.0, device=DEV)
    ys = torch.full((T + 1, H), -3.0, device=DEV)
    ws = torch.empty(m.moe_ffn_fp8_workspace_bytes(L, T, k), dtype=torch.uint8, device=DEV)
    m.moe_expert_ffn_fp8(L, r, T, k, yp[:T * k], q, d, ys[:T] if shared else None, ws)
    m.moe_check_device_errors()
    y, dy, sh, dsh = _reference(host, _codes(q), d.cpu().numpy(), r.idx.cpu().numpy())
    got = yp.double().cpu().numpy()
    assert (np.abs(got[:-1] - y) <= dy).all(), (np.abs(got[:-1] - y) / dy).max()
    assert (got[-1] == -3).all()
    if shared:
        got = ys.double().cpu().numpy()
        assert (np.abs(got[:-1] - sh) <= dsh).all()
        assert (got[-1] == -3).all()


@pytest.mark.parametrize("xt,flags", [("f32", 0), ("f16", 0), ("bf16", 0), ("bf16", 16), ("f32", 16)])
@pytest.mark.parametrize("T,E,k,H,I,shared", LAYERS)
def test_forward(T, E, k, H, I, shared, xt, flags):
    m = _qm()
    print("forward", xt, flags, T, E, k, H, I, shared, flush=True)
    g = np.random.default_rng(T * 3 + E + H)
    L, host = _layer(m, g, E, H, I, shared)
    lg = g.standard_normal((T, E)).astype(np.float32)
    bias = (0.05 * g.standard_normal(E)).astype(np.float32)
    kw = dict(score="sigmoid", scale=2.5)
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(DT[xt]).to(DEV)
    sc = torch.from_numpy(g.uniform(0.5, 1.5, T).astype(np.float32)).to(DEV) if shared else None
    out = torch.full((T + 1, H), -3.0, dtype=DT[xt], device=DEV)
    r = m.Routing(T, E, k, DEV)
    ws = torch.empty(m.moe_forward_fp8_workspace_bytes(L, T, k, flags), dtype=torch.uint8, device=DEV)
    m.moe_forward_fp8(L, torch.from_numpy(lg).to(DEV), x, k, r, m.RouteSpec(bias=torch.from_numpy(bias).to(DEV), **kw),
                      out[:T], sc, flags, ws)
    m.moe_check_device_errors()
    idx, w = ref.route(lg, k, bias=bias, **kw)
    assert np.array_equal(r.idx.cpu().numpy(), idx)
    q, d = _quantize(m, x)
    o, lim = _expected(host, _codes(q), d.cpu().numpy(), idx, w, sc, xt, flags)
    got = out.double().cpu().numpy()
    assert (np.abs(got[:-1] - o) <= lim).all(), (np.abs(got[:-1] - o) / lim).max()
    assert (got[-1] == -3).all()


@pytest.mark.parametrize("xt,flags", [("f32", 0), ("bf16", 16)])
@pytest.mark.parametrize("T,E,k,H,I,shared", [
    (2600, 8, 4, 2048, 1024, True),      # tiles of 128 tokens, several items a workgroup in both products
    (900, 64, 4, 1024, 512, True),       # of 64
    (1280, 40, 1, 512, 2048, False),     # of 32
    (1111, 2, 2, 1024, 1024, True),      # two long buckets
    (100, 2, 1, 8704, 128, False),       # rows longer than 64 scale blocks
    (17000, 4, 2, 512, 128, True),       # more tokens than one placing pass
    (70, 1024, 2, 512, 512, False),      # most experts without a token
])
def test_forward_long(T, E, k, H, I, shared, xt, flags):
    """Long calls against the reference at sampled tokens, with a hot expert and experts without a token."""
    m = _qm()
    print("forward long", xt, flags, T, E, k, H, I, shared, flush=True)
    g = np.random.default_rng(T + E + I)
    L, host = _layer(m, g, E, H, I, shared)
    lg = g.standard_normal((T, E)).astype(np.float32)
    lg[: T // 3, E // 2] += 4
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(DT[xt]).to(DEV)
    sc = torch.from_numpy(g.uniform(0.5, 1.5, T).astype(np.float32)).to(DEV) if shared else None
    out = torch.full((T + 1, H), -3.0, dtype=DT[xt], device=DEV)
    r = m.Routing(T, E, k, DEV)
    ws = torch.full((m.moe_forward_fp8_workspace_bytes(L, T, k, flags),), 0x7F, dtype=torch.uint8, device=DEV)
    m.moe_forward_fp8(L, torch.from_numpy(lg).to(DEV), x, k, r, m.RouteSpec(), out[:T], sc, flags, ws)
    m.moe_check_device_errors()
    at = np.unique(np.concatenate([[0, 1, T // 3 - 1, T // 3, T - 2, T - 1], g.integers(0, T, 40)]))
    idx, w = ref.route(lg[at], k)
    assert np.array_equal(r.idx.cpu().numpy()[at], idx)
    q, d = _quantize(m, x)
    o, lim = _expected(host, _codes(q)[at], d.cpu().numpy()[at], idx, w, sc[torch.from_numpy(at).to(DEV)] if shared else None, xt, flags)
    got = out.double().cpu().numpy()
    assert (np.abs(got[at] - o) <= lim).all(), (np.abs(got[at] - o) / lim).max()
    assert (got[-1] == -3).all() and np.isfinite(got).all()
    # every token: the same call once more, its tokens in reverse
    out2 = torch.empty_like(x)
    m.moe_forward_fp8(L, torch.from_numpy(lg[::-1].copy()).to(DEV), x.flip(0).contiguous(), k, r, m.RouteSpec(), out2,
                      sc.flip(0).contiguous() if shared else None, flags, ws)
    assert torch.equal(out2.flip(0), out[:T])


@pytest.mark.parametrize("T,H", [(40, 512), (300, 512), (300, 1024)])
def test_unaligned_token_scales(T, H):
    """xs needs 4-byte alignment only; the results are those of an aligned one, bit for bit in fp32."""
    m = _qm()
    g = np.random.default_rng(T)
    E, k, I = 4, 2, 512
    L, _ = _layer(m, g, E, H, I, True)
    r = m.Routing(T, E, k, DEV)
    m.moe_route_scored(torch.randn(T, E, device=DEV), k, r, m.RouteSpec(),
                       torch.empty(max(4, m.moe_route_workspace_bytes(T, E, k)), dtype=torch.uint8, device=DEV))
    q, d = _quantize(m, torch.randn(T, H, device=DEV))
    odd = torch.empty(d.numel() + 1, device=DEV)[1:].view(d.shape)
    odd.copy_(d)
    ws = torch.empty(m.moe_ffn_fp8_workspace_bytes(L, T, k), dtype=torch.uint8, device=DEV)
    res = []
    for s in (d, odd):
        yp, ys = torch.empty(T * k, H, device=DEV), torch.empty(T, H, device=DEV)
        m.moe_expert_ffn_fp8(L, r, T, k, yp, q, s, ys, ws)
        res += [yp, ys]
    m.moe_check_device_errors()
    assert torch.equal(res[0], res[2]) and torch.equal(res[1], res[3])


def test_forward_is_its_stages_and_repeats_bitwise():
    """moe_forward_fp8 equals route, quantise, expert FFN and combine called one after the other, in place and from
    dirty workspaces."""
    m = _qm()
    g = np.random.default_rng(12)
    for T, E, k, H, I in ((1, 16, 4, 512, 256), (50, 16, 4, 512, 256), (400, 16, 4, 512, 256)):
        L, _ = _layer(m, g, E, H, I, True)
        lg = torch.randn(T, E, device=DEV)
        x = torch.randn(T, H, device=DEV)
        spec = m.RouteSpec("sigmoid", 4, 2, 2, scale=1.5)
        r = m.Routing(T, E, k, DEV)
        rw = torch.empty(max(4, m.moe_route_workspace_bytes(T, E, k)), dtype=torch.uint8, device=DEV)
        m.moe_route_scored(lg, k, r, spec, rw)
        q, d = _quantize(m, x)
        yp, ys = torch.empty(T * k, H, device=DEV), torch.empty(T, H, device=DEV)
        m.moe_expert_ffn_fp8(L, r, T, k, yp, q, d, ys,
                             torch.empty(m.moe_ffn_fp8_workspace_bytes(L, T, k), dtype=torch.uint8, device=DEV))
        want = torch.empty(T, H, device=DEV)
        m.moe_combine(yp, r.w, want, ys)
        for fill in (0xFF, 0x7F):
            ws = torch.full((m.moe_forward_fp8_workspace_bytes(L, T, k),), fill, dtype=torch.uint8, device=DEV)
            xin = x.clone()
            m.moe_forward_fp8(L, lg, xin, k, m.Routing(T, E, k, DEV), spec, xin, workspace=ws)
            assert torch.equal(xin, want)
        m.moe_check_device_errors()


def test_a_token_does_not_depend_on_its_neighbours():
    m = _qm()
    g = np.random.default_rng(21)
    E, k, H, I, T = 8, 2, 256, 128, 200
    L, _ = _layer(m, g, E, H, I, False)
    lg, x = torch.randn(T, E, device=DEV), torch.randn(T, H, device=DEV).bfloat16()
    ws = torch.empty(m.moe_forward_fp8_workspace_bytes(L, T, k, 16), dtype=torch.uint8, device=DEV)
    out, out2 = torch.empty_like(x), torch.empty_like(x)
    m.moe_forward_fp8(L, lg, x, k, m.Routing(T, E, k, DEV), m.RouteSpec(), out, flags=16, workspace=ws)
    p = torch.randperm(T, device=DEV)
    m.moe_forward_fp8(L, lg[p].contiguous(), x[p].contiguous(), k, m.Routing(T, E, k, DEV), m.RouteSpec(), out2, flags=16,
                      workspace=ws)
    assert torch.equal(out[p], out2)


@pytest.mark.parametrize("T,H,I", [(40, 256, 128), (40, 512, 512), (600, 512, 512)])
def test_foreign_routing_buffers_raise_without_a_fault(T, H, I):
    """Counts, offsets and pair ids outside their range set the error word; nothing out of bounds is touched."""
    m = _qm()
    g = np.random.default_rng(2)
    E, k = 4, 2
    L, _ = _layer(m, g, E, H, I, False)
    q, d = _quantize(m, torch.randn(T, H, device=DEV))
    ws = torch.empty(m.moe_ffn_fp8_workspace_bytes(L, T, k), dtype=torch.uint8, device=DEV)
    yp = torch.zeros(T * k, H, device=DEV)
    for spoil in ("pair", "count", "offset"):
        r = m.Routing(T, E, k, DEV)
        m.moe_route_scored(torch.randn(T, E, device=DEV), k, r, m.RouteSpec(),
                           torch.empty(max(4, m.moe_route_workspace_bytes(T, E, k)), dtype=torch.uint8, device=DEV))
        t = getattr(r, spoil)
        t[1] = 1 << 20
        m.moe_expert_ffn_fp8(L, r, T, k, yp, q, d, workspace=ws)
        with pytest.raises(m.MoeError, match="out of range"):
            m.moe_check_device_errors()


def test_foreign_experts_of_few_pairs_raise_without_a_fault():
    """An expert index outside the layer sets the error word; the other pairs keep their results."""
    m = _qm()
    g = np.random.default_rng(3)
    T, E, k, H, I = 3, 16, 4, 256, 128
    L, _ = _layer(m, g, E, H, I, True)
    q, d = _quantize(m, torch.randn(T, H, device=DEV))
    ws = torch.empty(m.moe_ffn_fp8_workspace_bytes(L, T, k), dtype=torch.uint8, device=DEV)
    r = m.Routing(T, E, k, DEV)
    m.moe_route_scored(torch.randn(T, E, device=DEV), k, r, m.RouteSpec())
    want, ys = torch.empty(T * k, H, device=DEV), torch.empty(T, H, device=DEV)
    m.moe_expert_ffn_fp8(L, r, T, k, want, q, d, ys, ws)
    for bad in (E, -1, 1 << 30):
        r.idx[1, 2] = bad
        yp, y2 = torch.zeros(T * k, H, device=DEV), torch.empty(T, H, device=DEV)
        m.moe_expert_ffn_fp8(L, r, T, k, yp, q, d, y2, ws)
        with pytest.raises(m.MoeError, match="out of range"):
            m.moe_check_device_errors()
        keep = [p for p in range(T * k) if p != k + 2]
        assert torch.equal(yp[keep], want[keep]) and torch.equal(y2, ys)


def test_captured_layer_replays():
    """The layer captured in a graph, replayed with new inputs between eager work."""
    m = _qm()
    g = np.random.default_rng(31)
    for T, E, k, H, I in ((1, 16, 4, 512, 256), (90, 16, 4, 512, 256)):
        L, _ = _layer(m, g, E, H, I, True)
        lg, x = torch.randn(T, E, device=DEV), torch.randn(T, H, device=DEV).bfloat16()
        out, spec = torch.empty_like(x), m.RouteSpec("sigmoid", 4, 2, 2)
        r = m.Routing(T, E, k, DEV)
        ws = torch.empty(m.moe_forward_fp8_workspace_bytes(L, T, k, 16), dtype=torch.uint8, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            m.moe_forward_fp8(L, lg, x, k, r, spec, out, flags=16, workspace=ws)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.moe_forward_fp8(L, lg, x, k, r, spec, out, flags=16, workspace=ws)
        for _ in range(4):
            lg.normal_()
            x.normal_()
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            ws2 = torch.empty_like(ws)
            m.moe_forward_fp8(L, lg, x, k, m.Routing(T, E, k, DEV), spec, out, flags=16, workspace=ws2)
            assert torch.equal(got, out)
        m.moe_check_device_errors()


def test_two_streams_with_their_own_buffers():
    m = _qm()
    g = np.random.default_rng(41)
    T, E, k, H, I = 64, 16, 4, 512, 256
    L, _ = _layer(m, g, E, H, I, False)
    spec = m.RouteSpec()
    def work():
        lg, x = torch.randn(T, E, device=DEV), torch.randn(T, H, device=DEV)
        n = m.moe_forward_fp8_workspace_bytes(L, T, k)
        return lg, x, torch.empty_like(x), m.Routing(T, E, k, DEV), torch.empty(n, dtype=torch.uint8, device=DEV)
    sets = [work(), work()]
    want = []
    for lg, x, out, r, ws in sets:
        m.moe_forward_fp8(L, lg, x, k, r, spec, out, workspace=ws)
        want.append(out.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (lg, x, out, r, ws), s in zip(sets, streams):
            m.moe_forward_fp8(L, lg, x, k, r, spec, out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (_, _, out, _, _), w in zip(sets, want):
        assert torch.equal(out, w)
