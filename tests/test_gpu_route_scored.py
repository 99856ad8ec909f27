"""moe_route_scored against the 64-bit reference: experts, buckets and active lists
exact, weights within the rounding of one fp32 store."""
import numpy as np
import pytest

from tests import fp8_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda"


def _qm():
    import quantized_moe_ffn_amd as m
    m.load_library()
    return m


def _call(m, lg, k, spec, r=None, ws=None, stream=None):
    T, E = lg.shape
    r = r or m.Routing(T, E, k, DEV)
    ws = ws if ws is not None else torch.empty(max(m.moe_route_workspace_bytes(T, E, k), 4), dtype=torch.uint8, device=DEV)
    m.moe_route_scored(lg, k, r, spec, ws, stream)
    return r


def _check(r, logits, k, **kw):
    T, E = logits.shape
    idx, w = ref.route(logits, k, **kw)
    assert np.array_equal(r.idx.cpu().numpy(), idx)
    # fp64 scores (a few 2^-52 off), one rounding to fp32
    assert (np.abs(r.w.cpu().numpy() - w) <= np.abs(w) * (ref.U + 1e-12) + 1e-45).all()
    pair, count, offset, active = ref.buckets(idx, E)
    assert np.array_equal(r.pair.cpu().numpy(), pair)
    assert np.array_equal(r.count.cpu().numpy(), count) and np.array_equal(r.offset.cpu().numpy(), offset)
    n = int(r.n_active.item())
    assert n == len(active) and np.array_equal(r.active.cpu().numpy()[:n], active)


RULES = {
    "softmax": dict(score="softmax"),
    "softmax_raw": dict(score="softmax", renorm=False, scale=16.0),
    "sigmoid_bias": dict(score="sigmoid", bias=True, scale=2.5),
    "groups2": dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, bias=True),
    "groups1": dict(score="softmax", n_group=8, topk_group=3, group_top=1, renorm=False),
}


@pytest.mark.parametrize("rule", sorted(RULES))
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (1, 256, 8), (3, 512, 10), (7, 40, 3), (32, 256, 8), (33, 256, 8),
                                   (256, 64, 1), (257, 64, 1), (100, 72, 2), (777, 512, 10), (1000, 1024, 16),
                                   (4096, 256, 8)])
def test_matches_reference(rule, T, E, k):
    m = _qm()
    kw = dict(RULES[rule])
    if kw.get("n_group", 1) > 1 and k > kw["topk_group"] * (E // 8) or (E // kw.get("n_group", 1)) < kw.get("group_top", 1):
        pytest.skip("the groups hold fewer experts")
    print("route", rule, T, E, k, flush=True)
    g = np.random.default_rng(T * 7919 + E * 31 + k)
    lg = (g.standard_normal((T, E)) * 1.5 + 0.5 * g.standard_normal(E)).astype(np.float32)
    bias = (0.05 * g.standard_normal(E)).astype(np.float32) if kw.pop("bias", False) else None
    spec = m.RouteSpec(bias=None if bias is None else torch.from_numpy(bias).to(DEV), **kw)
    r = _call(m, torch.from_numpy(lg).to(DEV), k, spec)
    m.moe_check_device_errors()
    _check(r, lg, k, bias=bias, **kw)


def test_more_tokens_than_one_placing_pass():
    m = _qm()
    T, E, k = 16385, 64, 4
    lg = np.random.default_rng(5).standard_normal((T, E)).astype(np.float32)
    r = _call(m, torch.from_numpy(lg).to(DEV), k, m.RouteSpec("sigmoid", 8, 4, 2))
    m.moe_check_device_errors()
    _check(r, lg, k, score="sigmoid", n_group=8, topk_group=4, group_top=2)


@pytest.mark.parametrize("n_group,E", [(1, 64), (64, 64), (64, 128), (5, 100), (3, 33), (16, 1024), (7, 511)])
def test_group_counts(n_group, E):
    m = _qm()
    T, tg = 19, max(1, n_group // 2)
    S = E // n_group
    k = min(8, tg * S) if n_group > 1 else 8
    lg = np.random.default_rng(E + n_group).standard_normal((T, E)).astype(np.float32)
    for top in (1, 2)[:S]:
        r = _call(m, torch.from_numpy(lg).to(DEV), k, m.RouteSpec("sigmoid", n_group, tg, top))
        m.moe_check_device_errors()
        _check(r, lg, k, score="sigmoid", n_group=n_group, topk_group=tg, group_top=top)


def test_ties_go_to_the_lower_index_in_experts_and_groups():
    m = _qm()
    for E in (64, 200, 512, 1024):
        lg = np.zeros((5, E), np.float32)
        lg[1, 3::7] = 1.0
        lg[2] = np.where(np.arange(E) % 2, -0.0, 0.0)
        lg[3] = 50.0          # sigmoids that fp32 would round to one
        lg[3, E // 2] = 50.0 + 2.0 ** -18
        lg[4] = -200.0
        for kw in (dict(score="softmax"), dict(score="sigmoid"), dict(score="sigmoid", n_group=4, topk_group=2, group_top=2)):
            r = _call(m, torch.from_numpy(lg).to(DEV), 8, m.RouteSpec(**kw))
            m.moe_check_device_errors()
            _check(r, lg, 8, **kw)


def test_scores_that_only_64_bits_order():
    """Sigmoid scores 1e-9 apart order as their logits and biases do."""
    m = _qm()
    g = np.random.default_rng(3)
    lg = (18.0 + np.arange(64)[g.permutation(64)] * 2.0 ** -10).astype(np.float32)[None].repeat(4, 0)
    r = _call(m, torch.from_numpy(lg).to(DEV), 16, m.RouteSpec("sigmoid"))
    _check(r, lg, 16, score="sigmoid")


def test_barred_experts_and_sums_of_zero():
    m = _qm()
    E, k = 64, 4
    g = np.random.default_rng(8)
    lg = g.standard_normal((6, E)).astype(np.float32)
    lg[5] = -1e4                                   # every sigmoid is 0: weights 0, the lowest indices
    bias = np.zeros(E, np.float32)
    bias[::2] = -np.inf
    for kw in (dict(), dict(n_group=8, topk_group=2, group_top=2)):
        r = _call(m, torch.from_numpy(lg).to(DEV), k, m.RouteSpec("sigmoid", bias=torch.from_numpy(bias).to(DEV), **kw))
        m.moe_check_device_errors()
        _check(r, lg, k, score="sigmoid", bias=bias, **kw)
        assert (r.idx.cpu().numpy() % 2 == 1).all() and not r.w[5].any()
    bias[:] = -np.inf                              # nothing is left: the lowest indices, their own scores
    r = _call(m, torch.from_numpy(lg).to(DEV), k, m.RouteSpec("sigmoid", bias=torch.from_numpy(bias).to(DEV)))
    m.moe_check_device_errors()
    assert r.idx.cpu().tolist() == [[0, 1, 2, 3]] * 6


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_non_finite_logits_raise_and_stay_in_range(bad):
    m = _qm()
    for T in (5, 300):
        lg = np.random.default_rng(1).standard_normal((T, 256)).astype(np.float32)
        lg[3, 10:250] = bad
        for kw in (dict(score="softmax"), dict(score="sigmoid", n_group=8, topk_group=4, group_top=2)):
            r = _call(m, torch.from_numpy(lg).to(DEV), 8, m.RouteSpec(**kw))
            with pytest.raises(m.MoeError, match="non-finite router logit"):
                m.moe_check_device_errors()
            idx = r.idx.cpu().numpy()
            assert idx.min() >= 0 and idx.max() < 256 and all(len(set(row)) == 8 for row in idx)
            assert int(r.offset[-1]) == T * 8
    bias = torch.zeros(256, device=DEV)
    bias[7] = float("inf")
    _call(m, torch.zeros(2, 256, device=DEV), 8, m.RouteSpec("sigmoid", bias=bias))
    with pytest.raises(m.MoeError, match="non-finite router logit"):
        m.moe_check_device_errors()


def test_agrees_with_route_topk_on_plain_softmax():
    m = _qm()
    T, E, k = 100, 256, 8
    lg = torch.randn(T, E, device=DEV)
    a, b = m.Routing(T, E, k, DEV), m.Routing(T, E, k, DEV)
    ws = torch.empty(m.moe_route_workspace_bytes(T, E, k), dtype=torch.uint8, device=DEV)
    m.moe_route_topk(lg, k, a, True, ws)
    m.moe_route_scored(lg, k, b, m.RouteSpec(), ws)
    for n in ("idx", "count", "offset", "pair", "n_active"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    assert (a.w - b.w).abs().max().item() <= 1e-6
