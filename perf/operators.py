"""Cases of the scored routing, the 8-bit float quantiser, the block-scaled 8-bit
float matrix product and the mixture-of-experts layer over 8-bit float experts.

Each case carries the operator it runs in "op".  ``run`` computes it in its plain
form (elementary torch operations) where ``own`` is false, and with the library's
calls where it is true; ``exact`` is the definition in 64 bits.

Definitions, with e4m3 the 8-bit float with 4 exponent and 3 mantissa bits:
  route     s = softmax(l) or sigmoid(l) over the experts of a token; c = s + bias; with
            groups, only the experts of the topk_group groups with the largest group
            scores (sum of the group_top largest c of a group) stay; the k largest c
            are selected (ties to the lower index); w = s at them, divided by their sum
            (renorm), times scale; pairs bucketed by expert.
  quantize  per row and block of 128: a = max|x|; q = e4m3(x * 448 / a), d = a/448.
  matmul    y[t][n] = sum over blocks b of 128 of xs[t][b] * ws[n/128][b] *
            sum over j in b of xq[t][j] * wq[n][j].
  layer     route; x quantised; per selected expert h = silu(gate x) * (up x),
            h quantised, y = down h; out = sum of w * y (+ the shared expert's).
"""
import math

import torch

own = False

DEV = "cuda"
B = 128
E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}

# The layer shapes: the 256-expert / top-8 and the 512-expert / top-10 + shared
# ones of the block-quantized workloads and the tiny one, plus two of odd counts.
SAGE = {"H": 2048, "E": 256, "k": 8, "I": 512, "shared": False}
FLASH = {"H": 2560, "E": 512, "k": 10, "I": 512, "shared": True}
TINY = {"H": 256, "E": 8, "k": 2, "I": 256, "shared": False}
ODD_A = {"H": 1024, "E": 40, "k": 3, "I": 384, "shared": False}
ODD_B = {"H": 1280, "E": 96, "k": 6, "I": 640, "shared": True}

SOFTMAX = {"score": "softmax", "groups": 1, "topk_group": 1, "group_top": 1, "bias": False, "renorm": True, "scale": 1.0}
SIGMOID = {"score": "sigmoid", "groups": 1, "topk_group": 1, "group_top": 1, "bias": True, "renorm": True, "scale": 2.5}
GROUPED = {"score": "sigmoid", "groups": 8, "topk_group": 4, "group_top": 2, "bias": True, "renorm": True, "scale": 2.5}
GROUP_MAX = {"score": "softmax", "groups": 8, "topk_group": 3, "group_top": 1, "bias": False, "renorm": False, "scale": 16.0}


def listed():
    return [
        # one decoded token: balanced sigmoid routing over groups; latency
        {"name": "route_1", "op": "route", "T": 1, "E": 256, "k": 8, **GROUPED},
        # an odd batch of a prompt over 512 experts, softmax scores, no groups
        {"name": "route_777", "op": "route", "T": 777, "E": 512, "k": 10, **SOFTMAX},
        # a prompt chunk, balanced sigmoid routing over groups
        {"name": "route_4096", "op": "route", "T": 4096, "E": 256, "k": 8, **GROUPED},
        # a verify window's activations in fp32, then a prompt chunk's in bf16
        {"name": "quantize_3", "op": "quantize", "T": 3, "H": 2560, "x": "f32"},
        {"name": "quantize_4096", "op": "quantize", "T": 4096, "H": 2048, "x": "bf16"},
        # dense products next to the experts (a dense layer, a shared expert's projection)
        {"name": "matmul_1", "op": "matmul", "T": 1, "N": 2048, "K": 2560, "y": "bf16"},
        {"name": "matmul_333", "op": "matmul", "T": 333, "N": 1000, "K": 2000, "y": "f32"},
        {"name": "matmul_4096", "op": "matmul", "T": 4096, "N": 4096, "K": 4096, "y": "bf16"},
        # one decoded token, a verify-sized batch with a shared expert, an odd serving
        # batch and a prompt chunk through the whole layer
        {"name": "layer_1", "op": "layer", "T": 1, **SAGE, **GROUPED, "x": "bf16"},
        {"name": "layer_3_shared", "op": "layer", "T": 3, **FLASH, **SOFTMAX, "x": "bf16"},
        {"name": "layer_61", "op": "layer", "T": 61, **SAGE, **GROUPED, "x": "f16"},
        {"name": "layer_4096", "op": "layer", "T": 4096, **SAGE, **SIGMOID, "x": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "matmul", "matmul", "layer", "layer"])
    if op == "route":
        E, k = rng.randint(8, 512), rng.randint(1, 10)
        spec = dict(rng.choice([SOFTMAX, SIGMOID, GROUPED, GROUP_MAX]))
        if spec["groups"] > 1:
            E = max(24, E - E % 8)
            k = min(k, spec["topk_group"] * (E // 8))
        return {"op": op, "T": _log_int(rng, 1, 4096), "E": E, "k": min(k, E), **spec}
    if op == "quantize":
        return {"op": op, "T": _log_int(rng, 1, 4096), "H": 16 * rng.randint(16, 128), "x": rng.choice(["bf16", "f16", "f32"])}
    if op == "matmul":
        return {"op": op, "T": _log_int(rng, 1, 4096), "N": _log_int(rng, 64, 4096), "K": 16 * rng.randint(16, 256),
                "y": rng.choice(["bf16", "bf16", "f16", "f32"])}
    shape = dict(rng.choice([SAGE, FLASH, TINY, ODD_A, ODD_B]))
    spec = dict(rng.choice([SOFTMAX, SIGMOID, GROUPED]))
    top = SAGE["k"] * SAGE["H"] * SAGE["I"] / ((shape["k"] + shape["shared"]) * shape["H"] * shape["I"])
    T = _log_int(rng, 1, int(4096 * min(1.0, top)) // (2 if shape["E"] > 256 else 1))
    return {"op": op, "T": T, **shape, **(SIGMOID if shape["E"] == 8 else spec), "x": rng.choice(["bf16", "f16"])}


def _blocks(n):
    return (n + B - 1) // B


def _spec(case, g):
    """The routing rule a model's configuration holds, with its balance bias."""
    bias = torch.randn(case["E"], generator=g, device=DEV) * 0.05 if case["bias"] else None
    return {"bias": bias, **{n: case[n] for n in ("score", "groups", "topk_group", "group_top", "renorm", "scale")}}


def _logits(T, E, g):
    """Router logits: normal, with experts of different popularity."""
    return torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)


def _activations(T, H, dtype, g):
    """Rows of different size, with a few channels far larger than the others."""
    x = torch.randn(T, H, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    loud = 1.0 + 15.0 * (torch.rand(H, generator=g, device=DEV) < 0.01)
    return (x * loud).to(dtype)


def _weights(E, N, K, g):
    """Codes as a 128 x 128 block quantisation of normal weights leaves them, and the blocks' scales."""
    q = (torch.randn(E, N, K, generator=g, device=DEV) * 104.0).clamp_(-448.0, 448.0).to(E4M3)
    s = (0.5 + torch.rand(E, _blocks(N), _blocks(K), generator=g, device=DEV)) / (104.0 * math.sqrt(K))
    return q, s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, T = case["op"], case["T"]
    st = {"op": op}
    if op in ("route", "layer"):
        st.update(k=case["k"], spec=_spec(case, g), logits=_logits(T, case["E"], g))
    if op == "quantize":
        st["x"] = _activations(T, case["H"], DT[case["x"]], g)
    if op == "matmul":
        st["xq"], st["xs"] = _quantize(_activations(T, case["K"], torch.float32, g))
        wq, ws = _weights(1, case["N"], case["K"], g)
        st.update(wq=wq[0], ws=ws[0], y=DT[case["y"]])
    if op == "layer":
        H, E, I = case["H"], case["E"], case["I"]
        st["x"] = _activations(T, H, DT[case["x"]], g)
        mats = [("gate", E, I, H), ("up", E, I, H), ("down", E, H, I)]
        if case["shared"]:
            mats += [("sh_gate", 1, I, H), ("sh_up", 1, I, H), ("sh_down", 1, H, I)]
        for name, n, rows, cols in mats:
            st[name] = _weights(n, rows, cols, g)
        st["shared"] = case["shared"]
        # the capacity a caller of the plain form plans its padded buckets with
        st["rows"] = int(torch.bincount(_select(st["logits"], st["k"], st["spec"])[0].reshape(-1), minlength=E).max())
    if own:   # the handles and buffers a user's program keeps between calls
        import quantized_moe_ffn_amd as qm
        if op in ("route", "layer"):
            s = st["spec"]
            st["rule"] = qm.RouteSpec(score=s["score"], n_group=s["groups"], topk_group=s["topk_group"],
                                      group_top=s["group_top"], renorm=s["renorm"], scale=s["scale"], bias=s["bias"])
            st["routing"] = qm.Routing(T, case["E"], case["k"])
        if op == "route":
            n = qm.moe_route_workspace_bytes(T, case["E"], case["k"])
            st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
        if op == "quantize":
            st["out"] = (torch.empty((T, case["H"]), dtype=E4M3, device=DEV),
                         torch.empty((T, _blocks(case["H"])), dtype=torch.float32, device=DEV))
        if op == "matmul":
            st["matrix"] = qm.Fp8Matrix(st["wq"][None], st["ws"][None])
            st["out"] = torch.empty((T, case["N"]), dtype=st["y"], device=DEV)
        if op == "layer":
            m = {n: qm.Fp8Matrix(*st[n]) for n, *_ in mats}
            sh = (m["sh_gate"], m["sh_up"], m["sh_down"]) if case["shared"] else None
            st["layer"] = qm.Fp8Layer(m["gate"], m["up"], m["down"], sh)
            # bf16 outputs take the bf16 hand-off of the per-pair outputs, fp16 ones keep fp32
            st["flags"] = qm.MOE_FFN_PAIR_BF16 if case["x"] == "bf16" else 0
            n = qm.moe_forward_fp8_workspace_bytes(st["layer"], T, case["k"], st["flags"])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
            st["out"] = torch.empty_like(st["x"])
    return st


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import quantized_moe_ffn_amd as qm
    op = st["op"]
    if op == "route":
        qm.moe_route_scored(st["logits"], st["k"], st["routing"], st["rule"], st["ws"])
        r = st["routing"]
        return {"idx": r.idx, "w": r.w, "count": r.count, "offset": r.offset, "pair": r.pair}
    if op == "quantize":
        qm.moe_quantize_fp8(st["x"], *st["out"])
        return {"q": st["out"][0], "d": st["out"][1]}
    if op == "matmul":
        qm.moe_matmul_fp8(st["xq"], st["xs"], st["matrix"], st["out"])
        return st["out"]
    qm.moe_forward_fp8(st["layer"], st["logits"], st["x"], st["k"], st["routing"], st["rule"], st["out"],
                       flags=st["flags"], workspace=st["ws"])
    return {"out": st["out"], "idx": st["routing"].idx, "w": st["routing"].w}


# ------------------------------------------------------------------ the plain forms


def _select(logits, k, spec):
    """Selected experts and weights; scores next to a border need 64 bits to be ordered."""
    l = logits.double()
    s = torch.softmax(l, 1) if spec["score"] == "softmax" else torch.sigmoid(l)
    c = s if spec["bias"] is None else s + spec["bias"].double()
    if spec["groups"] > 1:
        cg = c.view(c.shape[0], spec["groups"], -1)
        gs = torch.topk(cg, spec["group_top"], dim=2).values.sum(2)
        best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :spec["topk_group"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, best, True)
        c = torch.where(keep[:, :, None], cg, -math.inf).view_as(c)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if spec["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx, (w * spec["scale"]).float()


def _buckets(idx, E):
    flat = idx.reshape(-1)
    pair = torch.sort(flat, stable=True).indices
    count = torch.zeros(E, dtype=torch.int64, device=idx.device).scatter_add_(0, flat, torch.ones_like(flat))
    offset = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    return pair, count, offset


def _quantize(x):
    """[T][K] -> codes and one scale for each 128 of a row."""
    T, K = x.shape
    xb = torch.nn.functional.pad(x.float(), (0, _blocks(K) * B - K)).view(T, -1, B)
    a = xb.abs().amax(2)
    v = xb * 448.0 / torch.where(a > 0, a, 1.0)[:, :, None]
    return v.to(E4M3).view(T, -1)[:, :K].contiguous(), a / 448.0


def _dequantize(q, d):
    T, K = q.shape
    return q.float() * d.repeat_interleave(B, 1)[:, :K]


def _dequantize_weights(q, s):
    """[E][N][K] codes and [E][N/128][K/128] scales -> fp32 weights."""
    return q.float() * s.repeat_interleave(B, 1)[:, :q.shape[1]].repeat_interleave(B, 2)[:, :, :q.shape[2]]


def _ffn(x, gate, up, down):
    """[E][n][H] rows through their experts' [E][I][H], [E][I][H], [E][H][I]."""
    g = torch.bmm(x, _dequantize_weights(*gate).transpose(1, 2).contiguous())
    u = torch.bmm(x, _dequantize_weights(*up).transpose(1, 2).contiguous())
    h = g * torch.sigmoid(g) * u
    h = _dequantize(*_quantize(h.view(-1, h.shape[2]))).view_as(h)
    return torch.bmm(h, _dequantize_weights(*down).transpose(1, 2).contiguous())


def _run_plain(st):
    op = st["op"]
    if op == "route":
        idx, w = _select(st["logits"], st["k"], st["spec"])
        pair, count, offset = _buckets(idx, st["logits"].shape[1])
        return {"idx": idx.int(), "w": w, "count": count.int(), "offset": offset.int(), "pair": pair.int()}
    if op == "quantize":
        q, d = _quantize(st["x"])
        return {"q": q, "d": d}
    if op == "matmul":
        w = _dequantize_weights(st["wq"][None], st["ws"][None])[0]
        return (_dequantize(st["xq"], st["xs"]) @ w.t()).to(st["y"])
    idx, w = _select(st["logits"], st["k"], st["spec"])
    T, k = idx.shape
    E, H = st["logits"].shape[1], st["x"].shape[1]
    x = _dequantize(*_quantize(st["x"]))
    if T * k <= E:   # few pairs: each with its own expert's matrices
        flat = idx.reshape(-1)
        y = _ffn(x.repeat_interleave(k, 0)[:, None], *[(q.view(torch.uint8)[flat].view(E4M3), s[flat]) for q, s in (st["gate"], st["up"], st["down"])])
        y = y.view(T, k, H)
    else:            # buckets padded to the fullest one
        pair, count, offset = _buckets(idx, E)
        e = idx.reshape(-1)[pair]
        slot = e * st["rows"] + torch.arange(T * k, device=DEV) - offset[e]
        xp = torch.zeros(E * st["rows"], H, device=DEV)
        xp[slot] = x[pair // k]
        yp = _ffn(xp.view(E, st["rows"], H), st["gate"], st["up"], st["down"]).view(-1, H)
        y = torch.empty(T * k, H, device=DEV)
        y[pair] = yp[slot]
        y = y.view(T, k, H)
    out = (w[:, :, None] * y).sum(1)
    if st["shared"]:
        out = out + _ffn(x[None], st["sh_gate"], st["sh_up"], st["sh_down"])[0]
    return {"out": out.to(st["x"].dtype), "idx": idx.int(), "w": w}


# ------------------------------------------------------------------ the definition in 64 bits


def _e4m3_64(v):
    """v rounded to the nearest e4m3 value, ties to even, in 64 bits (|v| at most 448)."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 4).clamp_min(-9))
    return torch.round(v / step) * step


def _quantize_64(x):
    T, K = x.shape
    codes, scales = torch.zeros_like(x), x.new_zeros(T, _blocks(K))
    for b in range(_blocks(K)):
        v = x[:, b * B:(b + 1) * B]
        a = v.abs().max(1, keepdim=True).values
        codes[:, b * B:(b + 1) * B] = torch.where(a > 0, _e4m3_64(v * 448 / a.clamp_min(1e-300)), 0.0)
        scales[:, b:b + 1] = a / 448
    return codes, scales


def _matmul_64(xq, xs, wq, ws):
    y = torch.zeros(xq.shape[0], wq.shape[0], dtype=torch.float64, device=xq.device)
    of_row = torch.arange(wq.shape[0], device=xq.device) // B
    for b in range(xs.shape[1]):
        part = xq[:, b * B:(b + 1) * B] @ wq[:, b * B:(b + 1) * B].t()
        y += part * xs[:, b:b + 1] * ws[of_row, b][None]
    return y


def _route_64(logits, k, spec):
    l = logits.double()
    if spec["score"] == "softmax":
        s = torch.exp(l - l.max(1, keepdim=True).values)
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-l))
    c = s.clone() if spec["bias"] is None else s + spec["bias"].double()
    T, E = c.shape
    rows = torch.arange(T, device=c.device)
    if spec["groups"] > 1:
        S = E // spec["groups"]
        left, score = c.clone(), torch.zeros(T, spec["groups"], dtype=torch.float64, device=c.device)
        for g in range(spec["groups"]):
            for _ in range(spec["group_top"]):
                m = left[:, g * S:(g + 1) * S].max(1)
                score[:, g] += m.values
                left[rows, g * S + m.indices] = -math.inf
        for _ in range(spec["groups"] - spec["topk_group"]):   # drop the lowest groups
            worst = (score.flip(1).argmin(1) - (spec["groups"] - 1)).neg()
            score[rows, worst] = math.inf
            for i in range(S):
                c[rows, worst * S + i] = -math.inf
    idx = torch.zeros(T, k, dtype=torch.int64, device=c.device)
    for j in range(k):
        idx[:, j] = (c == c.max(1, keepdim=True).values).to(torch.int32).argmax(1)
        c[rows, idx[:, j]] = -math.inf
    w = s.gather(1, idx)
    return idx, (w / w.sum(1, keepdim=True) if spec["renorm"] else w) * spec["scale"]


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "route":
        idx, w = _route_64(st["logits"], st["k"], st["spec"])
        return {"idx": idx, "w": w, "count": None, "offset": None, "pair": None}
    if st["op"] == "quantize":
        q, d = _quantize_64(st["x"].double())
        return {"q": q, "d": d}
    if st["op"] == "matmul":
        return _matmul_64(st["xq"].double(), st["xs"].double(), st["wq"].double(), st["ws"].double())
    idx, w = _route_64(st["logits"], st["k"], st["spec"])
    xq, xs = _quantize_64(st["x"].double())
    out = torch.zeros(st["x"].shape, dtype=torch.float64, device=DEV)

    def expert(rows, mats):
        g, u = (_matmul_64(xq[rows], xs[rows], q.double(), s.double()) for q, s in mats[:2])
        hq, hs = _quantize_64(g / (1 + torch.exp(-g)) * u)
        return _matmul_64(hq, hs, mats[2][0].double(), mats[2][1].double())

    for e in torch.unique(idx).tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        out.index_add_(0, t, w[t, j][:, None] * expert(t, [(st[n][0][e], st[n][1][e]) for n in ("gate", "up", "down")]))
    if st["shared"]:
        out += expert(slice(None), [(st[n][0][0], st[n][1][0]) for n in ("sh_gate", "sh_up", "sh_down")])
    return {"out": out, "idx": idx, "w": w}


def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        return {"bytes": T * case["E"] * 4 + T * case["k"] * 12 + case["E"] * 8, "flops": T * case["E"] * 8}
    if op == "quantize":
        H = case["H"]
        return {"bytes": T * H * (SIZE[case["x"]] + 1) + T * _blocks(H) * 4, "flops": 3 * T * H}
    if op == "matmul":
        N, K = case["N"], case["K"]
        return {"bytes": (T + N) * K + T * N * SIZE[case["y"]] + (T + _blocks(N)) * _blocks(K) * 4, "flops": 2 * T * N * K}
    H, E, I, k = case["H"], case["E"], case["I"], case["k"]
    touched = E * (1 - (1 - k / E) ** T) + case["shared"]
    return {"bytes": touched * 3 * H * I + T * H * 2 * SIZE[case["x"]] + T * E * 4, "flops": 6.0 * T * (k + case["shared"]) * H * I}
