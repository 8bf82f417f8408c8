"""The training step of a layer with 4-bit weights, in plain form and as the library's calls.

  linear   z = x W^T + b, y = act(z) + r with W in 4 bits; backward dz = dy act'(z), dx = dz W, db = sum over rows of dz
  gated    g = x Wg^T, u = x Wu^T, h = act(g) u with two 4-bit weights; backward dx = dg Wg + du Wu with
           dg = dh u act'(g), du = dh act(g)
  clip     norm = sqrt(sum of g^2 over all gradients), out = g min(1, max_norm / (norm + 1e-6))

W is the weight as it is dequantized into the compute dtype (code value times block constant, one binary32 product,
rounded to the dtype).  `run` computes one pass: with `own` false by elementary torch operations in binary32 (so it runs
without the library's operators), with `own` true through bit_optimizer_states_amd.binding.  `exact` is the definition
in binary64.
"""
import math

import torch

own = False

DEV = "cuda:0"
_DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}

# NF4: the 16 normal-quantile values, in code order; FP4: E2M1 over 6, sign in the highest bit
_NF4 = [-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
        -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
        0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045, 0.722956657409668, 1.0]
_FP4 = [v / 6.0 for v in (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)]
_FP4 = _FP4 + [-v for v in _FP4]


def _dyn8():
    """The signed dynamic code: decade e holds the 2^e bin midpoints of [0.1, 1] scaled by 10^(e-6); with their
    negatives, 0 and +1."""
    pos = sorted((2 ** (e + 1) + 18 * j + 9) / (2 ** (e + 1) * 10 ** (7 - e)) for e in range(7) for j in range(2 ** e))
    return [-v for v in reversed(pos)] + [0.0] + pos + [1.0]


def listed():
    """The cases that are always measured: the projections of a 7B decoder (4096 x 4096, 4096 x 11008) and its
    gradients, small batches, and ragged sizes."""
    nf4 = {"code": "nf4", "nested": True, "blocksize": 64, "dt": "bf16"}
    return [
        # one generated token: the down projection added to the residual stream
        {"name": "linear_decode_1", "op": "linear", "dir": "forward", "m": 1, "k": 11008, "n": 4096, **nf4,
         "bias": "", "act": "none", "residual": True, "keep": False},
        # a training batch of 2 x 2048 tokens through the same projection
        {"name": "linear_batch_4k", "op": "linear", "dir": "forward", "m": 4096, "k": 11008, "n": 4096, **nf4,
         "bias": "", "act": "none", "residual": True, "keep": False},
        # a short prompt through a small layer in binary16: odd rows and columns, everything in the epilogue
        {"name": "linear_ragged", "op": "linear", "dir": "forward", "m": 77, "k": 992, "n": 1001, "dt": "fp16",
         "code": "fp4", "nested": False, "blocksize": 128, "bias": "fp32", "act": "gelu", "residual": True,
         "keep": True},
        # the gradient of a projection with bias and activation, 2048 tokens
        {"name": "linear_grad_2k", "op": "linear", "dir": "backward", "m": 2048, "k": 4096, "n": 4096, **nf4,
         "bias": "fp32", "act": "gelu_tanh", "residual": False, "keep": True},
        # the gradient of a short sequence through an odd layer in binary32
        {"name": "linear_grad_ragged", "op": "linear", "dir": "backward", "m": 301, "k": 1056, "n": 2731,
         "dt": "fp32", "code": "nf4", "nested": False, "blocksize": 64, "bias": "fp32", "act": "silu",
         "residual": False, "keep": True},
        # eight sequences generating: both projections of the gated block
        {"name": "gated_decode_8", "op": "gated", "dir": "forward", "m": 8, "k": 4096, "n": 11008, **nf4,
         "act": "silu", "keep": False},
        # a training batch of 2 x 2048 tokens, both projections kept for the gradient
        {"name": "gated_batch_4k", "op": "gated", "dir": "forward", "m": 4096, "k": 4096, "n": 11008, **nf4,
         "act": "silu", "keep": True},
        # ... and its gradient
        {"name": "gated_grad_4k", "op": "gated", "dir": "backward", "m": 4096, "k": 4096, "n": 11008, **nf4,
         "act": "silu", "keep": True},
        # a prompt of 200 tokens, an odd inner size in binary16
        {"name": "gated_ragged", "op": "gated", "dir": "forward", "m": 200, "k": 1056, "n": 2731, "dt": "fp16",
         "code": "nf4", "nested": False, "blocksize": 128, "act": "gelu", "keep": False},
        # the gradients of an embedding table and two layers of a 7B decoder in bf16, over the limit
        {"name": "clip_layers", "op": "clip", "set": "layers", "count": 19, "n": 131072000, "dt": "bf16",
         "clips": True},
        # the gradients of low-rank adapters, 448 matrices of 4096 x 16 in binary32, over the limit
        {"name": "clip_adapters", "op": "clip", "set": "equal", "count": 448, "n": 65536, "dt": "fp32", "clips": True},
        # a few norm weights and biases of odd lengths, two types: latency; within the limit
        {"name": "clip_few", "op": "clip", "set": "ragged", "count": 12, "n": 4100, "dt": "mixed", "clips": False},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: 1 to 4096 rows, layers of 64 to 11008 inputs (a multiple of 32) and outputs (odd ones among
    them), every type, code and activation; sets of 1 to 500 gradients of 1 to 2^26 elements, 2^28 in all."""
    op, way = rng.choice([("linear", "forward"), ("linear", "backward"), ("gated", "forward"), ("gated", "backward"),
                          ("clip", "")])
    if op == "clip":
        count = _between(rng, 1, 500)
        return {"op": op, "set": rng.choice(["equal", "ragged"]), "count": count,
                "n": _between(rng, 1, min(1 << 26, (1 << 28) // count)), "dt": rng.choice(["fp32", "fp16", "bf16", "mixed"]),
                "clips": rng.random() < 0.6}
    dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    k, n = 32 * _between(rng, 2, 344), _between(rng, 64, 11008)
    if rng.random() < 0.5:
        n = (n + 63) // 64 * 64
    most = 4096 * 4096 * 11008 // (k * n) // (8 if dt == "fp32" else 1)
    case = {"op": op, "dir": way, "m": _between(rng, 1, max(1, min(4096, most))), "k": k, "n": min(n, 11008), "dt": dt,
            "code": rng.choice(["nf4", "nf4", "fp4"]), "nested": rng.random() < 0.5,
            "blocksize": rng.choice([64, 64, 128, 256, 4096])}
    if op == "gated":
        return {**case, "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]),
                "keep": way == "backward" or rng.random() < 0.5}
    act = rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"])
    return {**case, "bias": rng.choice(["", dt, "fp32"]), "act": act,
            "residual": way == "forward" and rng.random() < 0.5, "keep": way == "backward" or rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _normal(shape, g, std=1.0, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def _weight(c, g):
    """A weight [n, k] in 4 bits: codes, and the block constants, plain or nested."""
    total = c["n"] * c["k"]
    nb = -(-total // c["blocksize"])
    w = {"codes": torch.randint(0, 256, (total // 2,), dtype=torch.uint8, device=DEV, generator=g)}
    if c["nested"]:
        w["c2"] = torch.randint(0, 256, (nb,), dtype=torch.uint8, device=DEV, generator=g)
        w["absmax2"] = 0.004 + 0.004 * torch.rand(-(-nb // 256), device=DEV, generator=g)
        w["offset"] = torch.full((1,), 0.0475, device=DEV)
    else:
        w["absmax"] = 0.03 + 0.04 * torch.rand(nb, device=DEV, generator=g)
    return w


def _lengths(c):
    """Lengths of the gradients of a set."""
    count, n = c["count"], c["n"]
    if c["set"] == "equal":
        return [n] * count
    if c["set"] == "ragged":
        return [1 + (i * 2654435761 + 12345) % n for i in range(count)]
    # an embedding table of n elements in rows of 4096, then layers: four square projections, three of 4096 x 11008,
    # two norms
    layer = [4096 * 4096] * 4 + [4096 * 11008] * 3 + [4096] * 2
    return ([n] + layer * (count // len(layer) + 1))[:count]


def _types(c):
    """Types of the gradients of a set."""
    kinds = ["bf16", "fp32"] if c["dt"] == "mixed" else [c["dt"]]
    return [kinds[i % len(kinds)] for i in range(c["count"])]


def _prepare_clip(c, g):
    # the gradients of one type lie in one buffer, each at a multiple of 8 elements, as a training program's bucket
    # holds them
    s, lengths, types = {"case": c, "flat": {}, "out": {}}, _lengths(c), _types(c)
    views = []
    begin = dict.fromkeys(types, 0)
    for n, t in zip(lengths, types):
        views.append((t, begin[t], n))
        begin[t] += (n + 7) // 8 * 8
    total = 0.0
    for t in sorted(begin):
        flat = torch.zeros(begin[t], dtype=_DT[t], device=DEV)
        for kind, at, n in views:
            if kind == t:
                flat[at:at + n] = _normal(n, g, 1e-3 if t != "fp16" else 0.1, _DT[t])
                total += n * (1e-3 if t != "fp16" else 0.1) ** 2
        s["flat"][t], s["out"][t] = flat, torch.zeros_like(flat)
    s["out"]["norm"] = torch.zeros(1, device=DEV)
    s["max_norm"] = math.sqrt(total) * (0.3 if c["clips"] else 4.0)
    if own:
        # the table of the gradients' places, which a program builds once
        from bit_optimizer_states_amd import binding as qb
        s["table"] = qb.grad_table([(s["flat"][t][at:at + n], s["out"][t][at:at + n]) for t, at, n in views])
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, g)
    m, k, n, dt = case["m"], case["k"], case["n"], _DT[case["dt"]]
    s = {"case": case, "values": torch.tensor(_NF4 if case["code"] == "nf4" else _FP4, device=DEV),
         "dyn8": torch.tensor(_dyn8(), device=DEV), "w": _weight(case, g)}
    if case["op"] == "gated":
        s["w_up"] = _weight(case, g)
    # pre-activations of about unit size, gradients of a loss's size (binary16 with loss scaling)
    unit = 35.0 / math.sqrt(k)
    small = 1e-3 if case["dt"] != "fp16" else 0.1
    empty = lambda *shape: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
    if case["dir"] == "forward":
        chan = 0.5 + torch.rand(k, device=DEV, generator=g)
        s["x"] = (_normal((m, k), g, unit) * chan).to(dt)
        s["out"] = {"y": empty(m, n)}
        if case["op"] == "gated":
            if case["keep"]:
                s["out"].update(gate=empty(m, n), up=empty(m, n))
            return s
        s["bias"] = _normal(n, g, 0.5, _DT[case["bias"]]) if case["bias"] else None
        s["residual"] = _normal((m, n), g, 1.0, dt) if case["residual"] else None
        if case["keep"]:
            s["out"]["z"] = empty(m, n)
        return s
    s["dy"] = _normal((m, n), g, small, dt)
    s["out"] = {"dx": empty(m, k)}
    if case["op"] == "gated":
        s["gate"], s["up"] = _normal((m, n), g, 1.0, dt), _normal((m, n), g, 1.0, dt)
        return s
    s["z"] = _normal((m, n), g, 1.0, dt) if case["act"] != "none" else None
    if case["bias"]:
        s["out"]["dbias"] = torch.empty(n, dtype=_DT[case["bias"]], device=DEV)
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _scratch(size):
    return torch.empty(size, dtype=torch.uint8, device=DEV) if size else None


def _run_own(s):
    from bit_optimizer_states_amd import binding as qb
    c, out = s["case"], s["out"]
    if c["op"] == "clip":
        ws = _scratch(qb.qb_multi_tensor_grad_norm_workspace_bytes(c["count"]))
        qb.qb_multi_tensor_grad_norm(s["table"], c["count"], out["norm"], ws)
        qb.qb_multi_tensor_clip_grads(s["table"], c["count"], s["max_norm"], out["norm"])
        return out
    m, k, n, bs = c["m"], c["k"], c["n"], c["blocksize"]
    code = qb.QB_NF4 if c["code"] == "nf4" else qb.QB_FP4
    act = {"none": qb.QB_ACT_NONE, "relu": qb.QB_ACT_RELU, "gelu": qb.QB_ACT_GELU, "gelu_tanh": qb.QB_ACT_GELU_TANH,
           "silu": qb.QB_ACT_SILU}[c["act"]]
    xdt = {"fp32": qb.QB_F32, "fp16": qb.QB_F16, "bf16": qb.QB_BF16}[c["dt"]]
    parts = [(w["codes"], w.get("absmax"), qb.make_dq(w["c2"], w["absmax2"], w["offset"], 256) if c["nested"] else None)
             for w in ([s["w"], s["w_up"]] if c["op"] == "gated" else [s["w"]])]
    if c["op"] == "gated":
        gate, up = parts
        if c["dir"] == "forward":
            ws = _scratch(qb.qb_dequant_gated_workspace_bytes(xdt, m, k, n))
            qb.qb_dequant_gated(s["x"], gate, up, code, bs, n, out["y"], ws, act=act, gate_out=out.get("gate"),
                                up_out=out.get("up"))
        else:
            ws = _scratch(qb.qb_dequant_gated_backward_workspace_bytes(xdt, m, k, n))
            qb.qb_dequant_gated_backward(s["dy"], s["gate"], s["up"], gate, up, code, bs, k, out["dx"], ws, act=act)
        return out
    codes, absmax, dq = parts[0]
    if c["dir"] == "forward":
        ws = _scratch(qb.qb_dequant_linear_workspace_bytes(xdt, m, k, n))
        qb.qb_dequant_linear(s["x"], codes, absmax, code, bs, n, out["y"], ws, bias=s["bias"], act=act,
                             residual=s["residual"], z=out.get("z"), dq=dq)
    else:
        ws = _scratch(qb.qb_dequant_linear_backward_workspace_bytes(xdt, m, k, n))
        qb.qb_dequant_linear_backward(s["dy"], codes, absmax, code, bs, k, out["dx"], ws, act=act, z=s["z"],
                                      dbias=out.get("dbias"), dq=dq)
    return out


# ---------------------------------------------------------------------------
# the plain forms, in binary32
# ---------------------------------------------------------------------------

def _dequant(s, w):
    """The weight [n, k] as the compute dtype holds it, in binary32."""
    c = s["case"]
    byte = w["codes"].int()
    code = torch.stack([byte >> 4, byte & 15], dim=1).view(-1)
    a = s["dyn8"][w["c2"].int()] * w["absmax2"].repeat_interleave(256)[:w["c2"].numel()] + w["offset"] \
        if c["nested"] else w["absmax"]
    v = s["values"][code] * a.repeat_interleave(c["blocksize"])[:code.numel()]
    return v.to(_DT[c["dt"]]).float().view(c["n"], c["k"])


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(kind, z):
    if kind == "none":
        return z
    if kind == "relu":
        return z.clamp_min(0.0)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if kind == "gelu_tanh":
        return z * _sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
    return z * _sigmoid(z)


def _act_grad(kind, z):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0.0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        a = 2.0 * math.sqrt(2.0 / math.pi)
        p, q = _sigmoid(a * (z + 0.044715 * z * z * z)), _sigmoid(-a * (z + 0.044715 * z * z * z))
        return p + z * p * q * a * (1.0 + 3.0 * 0.044715 * z * z)
    return _sigmoid(z) * (1.0 + z * _sigmoid(-z))


def _run_plain(s):
    c = s["case"]
    if c["op"] == "clip":
        norm = sum((f.float() * f.float()).sum(dtype=torch.float64) for f in s["flat"].values()).sqrt()
        scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
        return {**{t: (f.float() * scale).to(f.dtype) for t, f in s["flat"].items()}, "norm": norm.float().view(1)}
    dt = _DT[c["dt"]]
    w = _dequant(s, s["w"])
    if c["op"] == "gated":
        w_up = _dequant(s, s["w_up"])
        if c["dir"] == "forward":
            g, u = s["x"].float() @ w.T, s["x"].float() @ w_up.T
            kept = {"gate": g.to(dt), "up": u.to(dt)} if c["keep"] else {}
            return {"y": (_act(c["act"], g) * u).to(dt), **kept}
        dh, g, u = s["dy"].float(), s["gate"].float(), s["up"].float()
        return {"dx": ((dh * u * _act_grad(c["act"], g)) @ w + (dh * _act(c["act"], g)) @ w_up).to(dt)}
    if c["dir"] == "forward":
        z = s["x"].float() @ w.T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(c["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), **({"z": z.to(dt)} if c["keep"] else {})}
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(c["act"], s["z"].float())
    sums = {"dbias": dz.sum(0).to(_DT[c["bias"]])} if c["bias"] else {}
    return {"dx": (dz @ w).to(dt), **sums}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the work that a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "clip":
        size = sum(n * _SIZE[t] for n, t in zip(_lengths(case), _types(case)))
        return {"bytes": 2 * size + 4, "flops": 3 * sum(_lengths(case))}
    m, k, n, e = case["m"], case["k"], case["n"], _SIZE[case["dt"]]
    count = 2 if case["op"] == "gated" else 1
    weights = count * n * k * (0.5 + (1.0 if case["nested"] else 4.0) / case["blocksize"])
    flops = 2 * count * m * k * n
    if case["op"] == "gated":
        arrays = (3 if case["keep"] else 1) * m * n * e
    elif case["dir"] == "forward":
        arrays = (1 + case["residual"] + case["keep"]) * m * n * e
    else:
        arrays = (2 if case["act"] != "none" else 1) * m * n * e
    bias = n * _SIZE[case["bias"]] if case.get("bias") else 0
    return {"bytes": int(weights + arrays + m * k * e + bias), "flops": flops}


# ---------------------------------------------------------------------------
# the definition in binary64
# ---------------------------------------------------------------------------

def _exact_weight(c, w):
    """The weight in binary64: binary32 operations up to the compute dtype, whose value it is by definition."""
    element = torch.arange(c["n"] * c["k"], device=DEV)
    nibble = (w["codes"][element // 2] >> (4 - 4 * (element % 2)).to(torch.uint8)) & 15
    block = torch.div(element, c["blocksize"], rounding_mode="floor")
    if c["nested"]:
        table = torch.tensor(_dyn8(), dtype=torch.float32, device=DEV)
        constant = torch.add(torch.mul(table[w["c2"].long()], w["absmax2"][torch.arange(w["c2"].numel(), device=DEV) // 256]),
                             w["offset"])
    else:
        constant = w["absmax"]
    table = torch.tensor(_NF4 if c["code"] == "nf4" else _FP4, dtype=torch.float32, device=DEV)
    value = torch.mul(table[nibble.long()], constant[block])
    return value.to(_DT[c["dt"]]).reshape(c["n"], c["k"]).double()


def _exact_act(kind, z):
    """act(z) and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        on = torch.where(z > 0, 1.0, 0.0).double()
        return on * z, on
    if kind == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(z.square() / -2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        inner = math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
        t = torch.tanh(inner)
        return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t.square()) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z.square())
    p = torch.special.expit(z)
    return z * p, p + z * p * (1 - p)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        square = 0.0
        for flat in s["flat"].values():
            square = square + sum(part.double().pow(2).sum() for part in flat.split(1 << 26))
        norm = torch.sqrt(square)
        scale = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return {**{t: flat.double().mul_(scale) for t, flat in s["flat"].items()}, "norm": norm.reshape(1)}
    w = _exact_weight(case, s["w"])
    if case["op"] == "gated":
        w_up = _exact_weight(case, s["w_up"])
        if case["dir"] == "forward":
            x = s["x"].double()
            g, u = torch.mm(x, w.t()), torch.mm(x, w_up.t())
            return {"y": _exact_act(case["act"], g)[0] * u, **({"gate": g, "up": u} if case["keep"] else {})}
        a, slope = _exact_act(case["act"], s["gate"].double())
        dh = s["dy"].double()
        return {"dx": torch.mm(slope.mul_(s["up"].double()).mul_(dh), w) + torch.mm(a.mul_(dh), w_up)}
    if case["dir"] == "forward":
        z = torch.mm(s["x"].double(), w.t())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(case["act"], z)[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, **({"z": z} if case["keep"] else {})}
    dz = s["dy"].double()
    if s["z"] is not None:
        dz = dz * _exact_act(case["act"], s["z"].double())[1]
    return {"dx": torch.mm(dz, w), **({"dbias": dz.sum(0)} if case["bias"] else {})}
