"""Pins of the 64-bit reference of the 8-bit float operators (CPU)."""
import numpy as np
import pytest

from tests import fp8_ref as ref

torch = pytest.importorskip("torch")


def test_code_table_is_torchs_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3, equal_nan=True)


def test_encode_rounds_to_nearest_even_code():
    v = np.random.default_rng(0).uniform(-448, 448, 4096) * 2.0 ** np.random.default_rng(1).integers(-16, 1, 4096)
    v = np.concatenate([v, ref._MID, -ref._MID, ref._POS, [0.0, -0.0]])
    got = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(v), got)


def test_quantize_spans_the_format_and_zero_blocks_stay_zero():
    x = np.random.default_rng(2).standard_normal((3, 300))
    x[1, 128:256] = 0
    q, d = ref.quantize(x)
    assert d.shape == (3, 3) and d[1, 1] == 0 and not q[1, 128:256].any()
    assert np.abs(ref.decode(q[0, :128])).max() == 448
    err = np.abs(ref.dequant_x(q, d) - x)
    a = np.repeat(d * 448, 128, 1)[:, :300]
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, a / 448 * 2.0 ** -10) * (1 + 1e-12)).all()


def test_groups_limit_the_selection():
    l = np.array([[9.0, 1, 1, 1, 5, 5, 5, 5]])
    assert ref.route(l, 2)[0].tolist() == [[0, 4]]
    assert ref.route(l, 2, "sigmoid", n_group=2, topk_group=1, group_top=2)[0].tolist() == [[4, 5]]
    assert ref.route(l, 2, "sigmoid", n_group=2, topk_group=1, group_top=1)[0].tolist() == [[0, 1]]
    idx, w = ref.route(l, 3, "sigmoid", bias=[-1.0, 0, 0, 0, 0, 0, 0, 0], scale=2.5)
    assert idx.tolist() == [[4, 5, 6]] and abs(w.sum() - 2.5) < 1e-12
