"""Operators around a mixture-of-experts layer whose experts are the caller's own
or hold 4-bit weights, as workloads that can be timed and checked: the rows of a
batch sorted by expert (`dispatch`) and weighted back (`combine`), both with
their gradients, products with 4-bit weights and group scales (`w4`), the same
by expert (`grouped`), and the layer that these make together (`layer`).

`run` computes one pass in plain torch operations, or, where `own` is true,
through the library's entry points. Conventions:
  * slot t * k + j is the j-th choice of token t. Rows are grouped by expert,
    within an expert by slot; inv is a slot's row, pair a row's slot, offsets
    the experts' first rows. A slot whose expert is outside [0, experts), as on
    a device that holds a share of the experts, has no row: inv is -1, and the
    rows behind the last expert's stay as they were (pair is -1 there).
  * a weight is (q - z) * s: q four bits, two columns a byte, the even column
    low; s one scale per output feature and group of columns, z its zero point,
    a byte (8 without).
"""
import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROW_WEIGHTS = 1 << 30  # the plain products by expert gather weights by row up to here


def listed():
    return [
        # -- rows to their experts --
        # one new token on the 512-expert layer
        {"name": "dispatch_one_token", "op": "dispatch", "tokens": 1, "hidden": 4096,
         "experts": 512, "k": 10, "type": "bf16", "share": 1},
        # a packed prompt on a device that holds a quarter of 128 experts, in fp32, with a
        # row length that fills no power of two
        {"name": "dispatch_share", "op": "dispatch", "tokens": 3001, "hidden": 1000,
         "experts": 32, "k": 8, "type": "f32", "share": 4},
        # the gradient of a training batch's rows on the 512-expert layer, the largest
        {"name": "dispatch_gradient", "op": "dispatch_gradient", "tokens": 4096, "hidden": 4096,
         "experts": 512, "k": 10, "type": "bf16", "share": 1},
        # -- and back --
        # a decode batch on the 128-expert layer, fp32 rows
        {"name": "combine_decode_batch", "op": "combine", "tokens": 48, "hidden": 2048,
         "experts": 128, "k": 8, "type": "f32", "out": "bf16", "share": 1, "shared": False},
        # a prompt on the 512-expert layer with its shared expert
        {"name": "combine_prompt", "op": "combine", "tokens": 4096, "hidden": 4096,
         "experts": 512, "k": 10, "type": "bf16", "out": "bf16", "share": 1, "shared": True},
        # the gradients of rows and gates of a training batch on the 128-expert layer
        {"name": "combine_gradient", "op": "combine_gradient", "tokens": 4099, "hidden": 2048,
         "experts": 128, "k": 8, "type": "bf16", "out": "bf16", "share": 1},
        # -- products with 4-bit weights --
        # one new token through a projection
        {"name": "w4_one_token", "op": "w4", "rows": 1, "n": 4096, "k": 2048, "group": 128,
         "scales": "bf16", "zeros": False, "bias": False, "out": "bf16", "swiglu": False,
         "strided": False},
        # a short prompt, rows taken out of a wider buffer, small groups with zero points, a
        # bias, fp32 output
        {"name": "w4_short_prompt", "op": "w4", "rows": 77, "n": 2112, "k": 4096, "group": 32,
         "scales": "f32", "zeros": True, "bias": True, "out": "f32", "swiglu": False,
         "strided": True},
        # a long prompt through the widest projection
        {"name": "w4_long_prompt", "op": "w4", "rows": 4096, "n": 8192, "k": 4096, "group": 128,
         "scales": "f32", "zeros": False, "bias": False, "out": "bf16", "swiglu": False,
         "strided": False},
        # -- by expert --
        # gate and up of a decode batch of 8 on the 512-expert layer
        {"name": "grouped_decode_batch", "op": "grouped", "tokens": 8, "experts": 512, "k": 10,
         "n": 2048, "cols": 4096, "group": 128, "scales": "bf16", "zeros": False, "out": "bf16",
         "swiglu": True, "share": 1},
        # gate and up of a prompt on the 128-expert layer
        {"name": "grouped_prompt", "op": "grouped", "tokens": 4096, "experts": 128, "k": 8,
         "n": 1536, "cols": 2048, "group": 64, "scales": "bf16", "zeros": True, "out": "bf16",
         "swiglu": True, "share": 1},
        # -- the whole run of them: a decode batch through the 128-expert layer --
        {"name": "layer_decode_batch", "op": "layer", "tokens": 16, "experts": 128, "k": 8,
         "hidden": 2048, "inter": 768, "group": 128, "scales": "bf16", "zeros": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _drawn(rng):
    op = rng.choice(["dispatch", "dispatch_gradient", "combine", "combine_gradient", "w4", "w4",
                     "w4", "grouped", "grouped", "layer"])
    group = rng.choice([32, 64, 128])
    weights = {"group": group, "scales": rng.choice(["bf16", "f32"]), "zeros": rng.random() < 0.5}
    out = rng.choice(["bf16", "f32"])
    if op == "w4":
        n = _log_int(rng, 32, 8192)
        return {"op": op, "rows": _log_int(rng, 1, 8192), "n": n + n % 2,
                "k": group * _log_int(rng, 1, 8192 // group), **weights,
                "bias": rng.random() < 0.3, "out": out, "swiglu": rng.random() < 0.3,
                "strided": rng.random() < 0.3}
    experts = _log_int(rng, 2, 512)
    k = rng.randint(1, min(16, experts))
    share = rng.choice([1, 1, 2, 4])
    if op == "grouped" or op == "layer":
        case = {"op": op, "tokens": _log_int(rng, 1, 4096), "experts": experts, "k": k, **weights}
        cols = group * _log_int(rng, max(1, 256 // group), 4096 // group)
        n = group * _log_int(rng, max(1, 256 // group), 2048 // group)
        if op == "layer":
            return {**case, "hidden": cols, "inter": n}
        return {**case, "n": n, "cols": cols, "swiglu": rng.random() < 0.5, "share": share,
                "out": out}
    hidden = _log_int(rng, 16, 8192)
    case = {"op": op, "tokens": _log_int(rng, 1, 16384),
            "hidden": hidden + (-hidden) % rng.choice([1, 2, 8, 64]), "experts": experts, "k": k,
            "type": rng.choice(["bf16", "f32"]), "share": share}
    if op == "combine" or op == "combine_gradient":
        case["out"] = out
    if op == "combine":
        case["shared"] = rng.random() < 0.3
    return case


def draw(rng):
    most = {m: max(work(case)[m] for case in listed()) for m in ("bytes", "flops")}
    while True:
        case = _drawn(rng)
        bank = case["experts"] * max(case.get("n", 0) * case.get("cols", 0),
                                     2 * case.get("inter", 0) * case.get("hidden", 0)) \
            if "group" in case and "experts" in case else 0
        if all(work(case)[m] <= most[m] for m in most) and bank <= 1 << 29:
            return case


# ------------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 11)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _choices(g, case):
    """Each token's k experts, some experts liked more, and its gates. On a device
    with a share of the experts the ids count from its own first one."""
    t, k, share = case["tokens"], case["k"], case.get("share", 1)
    e = case["experts"] * share
    top, idx = (_randn(g, t, e) + 0.4 * _randn(g, e)).topk(k, dim=1)
    first = (share - 1) // 2 * case["experts"]
    return (idx - first).to(torch.int32), torch.softmax(top, dim=1)


def _activations(g, rows, cols):
    """N(0, 1) with a few large columns, as a normalised residual stream has."""
    x = _randn(g, rows, cols)
    big = torch.rand(cols, generator=g, device=DEV) < 0.01
    return torch.where(big, x * 12.0, x).to(torch.bfloat16)


def _weights(g, shape, case):
    """4-bit weights of `shape` [..., n, k]: codes heaped around the middle, as
    quantised weights are, scales with a spread, zero points about 8."""
    *head, n, k = shape
    group = case["group"]
    def nibble():
        def draw(hi):
            return torch.randint(0, hi, (*head, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        return draw(6).add_(draw(6)).add_(draw(6))
    codes = nibble().add_(nibble().mul_(16))
    s = torch.exp2(torch.randint(-8, 9, (*head, n, k // group), generator=g, device=DEV).float() / 8.0)
    s = (s * 0.02 / math.sqrt(8.0)).to(TYPES[case["scales"]])
    z = None
    if case["zeros"]:
        z = torch.randint(5, 12, (*head, n, k // group), generator=g, device=DEV, dtype=torch.uint8)
    return codes, s, z


def _indexes(idx, experts):
    """(experts of the rows, offsets, pair, inv): a stable sort of the slots."""
    flat = idx.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    ranked, order = torch.sort(key, stable=True)
    place = torch.arange(flat.numel(), device=flat.device)
    offsets = torch.searchsorted(ranked, torch.arange(experts + 1, device=flat.device))
    pair = torch.where(ranked < experts, order, -1)
    inv = torch.empty_like(place).scatter_(0, order, place)
    inv = torch.where(key < experts, inv, -1).view(idx.shape)
    return ranked, offsets.to(torch.int32), pair.to(torch.int32), inv.to(torch.int32)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "w4":
        m, k = case["rows"], case["k"]
        wide = k + 64 if case["strided"] else k
        s["x"] = _activations(g, m, wide)[:, :k]
        s["w"], s["ws"], s["wz"] = _weights(g, (case["n"], k), case)
        s["bias"] = _randn(g, case["n"]) if case["bias"] else None
        return s
    s["idx"], s["gates"] = _choices(g, case)
    ranked, s["offsets"], s["pair"], s["inv"] = _indexes(s["idx"], case["experts"])
    t, p = case["tokens"], case["tokens"] * case["k"]
    if op == "layer":
        h, i = case["hidden"], case["inter"]
        s["x"] = _activations(g, t, h)
        s["w1"] = _weights(g, (case["experts"], 2 * i, h), case)
        s["w2"] = _weights(g, (case["experts"], h, i), case)
        s["most"] = max(1, int(s["offsets"].diff().max()))
        return s
    if op == "grouped":
        s["x"] = _activations(g, p, case["cols"])
        s["w"] = _weights(g, (case["experts"], case["n"], case["cols"]), case)
        s["most"] = max(1, int(s["offsets"].diff().max()))
        n = case["n"] // 2 if case["swiglu"] else case["n"]
        s["buffer"] = torch.zeros(p, n, device=DEV, dtype=TYPES[case["out"]])
        return s
    h, kind = case["hidden"], TYPES[case["type"]]
    if op == "dispatch":
        s["x"] = _randn(g, t, h).to(kind)
    else:
        s["rows"] = _randn(g, p, h).to(kind)
    if op == "combine":
        s["shared"] = _randn(g, t, h).to(kind) if case["shared"] else None
    if op == "combine_gradient":
        s["d_out"] = _randn(g, t, h).to(TYPES[case["out"]])
    if op in ("dispatch", "combine_gradient"):
        s["buffer"] = torch.zeros(p, h, device=DEV, dtype=kind)
    return s


# --------------------------------------------------------------- plain forms --
def _dispatch(x, idx, experts):
    ranked, offsets, pair, inv = _indexes(idx, experts)
    rows = x[pair.clamp(min=0).long() // idx.shape[1]]
    return torch.where((ranked < experts)[:, None], rows, 0), offsets, pair, inv


def _by_token(rows, inv, weight, more, out):
    v = rows[inv.clamp(min=0).long()].float()  # [T][k][H]
    v = torch.where((inv >= 0)[:, :, None], v, 0.0)
    y = v.sum(dim=1) if weight is None else (v * weight[:, :, None]).sum(dim=1)
    return (y if more is None else y + more.float()).to(out)


def _combine_gradient(d_out, rows, gates, inv, pair):
    d = d_out.float()
    slot = pair.clamp(min=0).long()
    weight = torch.where(pair >= 0, gates.reshape(-1)[slot], 0.0)
    d_rows = (weight[:, None] * d[slot // gates.shape[1]]).to(rows.dtype)
    v = torch.where((inv >= 0)[:, :, None], rows[inv.clamp(min=0).long()].float(), 0.0)
    return d_rows, (v * d[:, None, :]).sum(dim=2)


def _values(w, ws, wz, kind=torch.float32):
    """What 4-bit weights [..., n, k / 2] stand for."""
    q = torch.stack((w & 15, w >> 4), dim=-1).flatten(-2).to(kind)
    group = q.shape[-1] // ws.shape[-1]
    q = q.unflatten(-1, (-1, group))
    zero = 8.0 if wz is None else wz[..., None].to(kind)
    return ((q - zero) * ws[..., None].to(kind)).flatten(-2)


def _activated(y, swiglu):
    if not swiglu:
        return y
    gate, up = y.chunk(2, dim=-1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _product(x, w, ws, wz, bias, swiglu, out):
    y = x.float() @ _values(w, ws, wz).t()
    if bias is not None:
        y = y + bias
    return _activated(y, swiglu).to(out)


def _grouped(x, offsets, w, most, swiglu, out):
    """Rows of x sorted by expert times their experts' weights: each row's own
    weights gathered where that is little, else all experts at once with the
    rows padded to the longest expert's."""
    p, e = x.shape[0], w[0].shape[0]
    row = torch.arange(p, device=x.device)
    expert = torch.searchsorted(offsets[1:].long(), row, right=True)
    valid = (expert < e)[:, None]
    expert = expert.clamp(max=e - 1)
    if p * w[0].shape[1] * x.shape[1] <= ROW_WEIGHTS:
        mine = _values(*(None if v is None else v[expert] for v in w))
        y = torch.matmul(mine, x.float()[:, :, None])[:, :, 0]
    else:
        first = offsets[:-1].long()
        at = (first[:, None] + torch.arange(most, device=x.device)).clamp(max=p - 1)
        y = torch.matmul(_values(*w), x.float()[at].transpose(1, 2).contiguous())
        y = y[expert, :, (row - first[expert]).clamp(max=most - 1)]
    return torch.where(valid, _activated(y, swiglu), 0.0).to(out)


def _plain(s, case):
    op = case["op"]
    if op == "dispatch":
        return _dispatch(s["x"], s["idx"], case["experts"])
    if op == "dispatch_gradient":
        return _by_token(s["rows"], s["inv"], None, None, s["rows"].dtype)
    if op == "combine":
        return _by_token(s["rows"], s["inv"], s["gates"], s["shared"], TYPES[case["out"]])
    if op == "combine_gradient":
        return _combine_gradient(s["d_out"], s["rows"], s["gates"], s["inv"], s["pair"])
    if op == "w4":
        return _product(s["x"], s["w"], s["ws"], s["wz"], s["bias"], case["swiglu"],
                        TYPES[case["out"]])
    if op == "grouped":
        return _grouped(s["x"], s["offsets"], s["w"], s["most"], case["swiglu"],
                        TYPES[case["out"]])
    rows, offsets, _, inv = _dispatch(s["x"], s["idx"], case["experts"])
    h = _grouped(rows, offsets, s["w1"], s["most"], True, torch.bfloat16)
    y = _grouped(h, offsets, s["w2"], s["most"], False, torch.bfloat16)
    return _by_token(y, inv, s["gates"], None, torch.bfloat16)


# ---------------------------------------------------------------------- run --
def run(state):
    s, case = state, state["case"]
    if not own:
        return _plain(s, case)
    import block_fp8_routed_amd as moe
    op = case["op"]
    if op == "dispatch":
        return moe.moe_dispatch(s["x"], s["idx"], case["experts"], out=s["buffer"])
    if op == "dispatch_gradient":
        return moe.moe_dispatch_backward(s["rows"], s["inv"])
    if op == "combine":
        return moe.moe_combine(s["rows"], s["gates"], s["inv"], shared=s["shared"],
                               out_dtype=TYPES[case["out"]])
    if op == "combine_gradient":
        return moe.moe_combine_backward(s["d_out"], s["rows"], s["gates"], s["inv"],
                                        out=s["buffer"])
    if op == "w4":
        return moe.moe_linear_w4(s["x"], s["w"], s["ws"], s["wz"], bias=s["bias"],
                                 swiglu=case["swiglu"], out_dtype=TYPES[case["out"]])
    if op == "grouped":
        return moe.moe_grouped_linear_w4(s["x"], s["offsets"], *s["w"], swiglu=case["swiglu"],
                                         out=s["buffer"])
    rows, offsets, _, inv = moe.moe_dispatch(s["x"], s["idx"], case["experts"])
    h = moe.moe_grouped_linear_w4(rows, offsets, *s["w1"], swiglu=True)
    y = moe.moe_grouped_linear_w4(h, offsets, *s["w2"])
    return moe.moe_combine(y, s["gates"], inv)


def _weight_bytes(n, k, case):
    size = 2 if case["scales"] == "bf16" else 4
    return n * k // 2 + n * (k // case["group"]) * (size + (1 if case["zeros"] else 0))


def work(case):
    op = case["op"]
    if op == "w4":
        m, n, k = case["rows"], case["n"], case["k"]
        n_out = n // 2 if case["swiglu"] else n
        return {"bytes": m * k * 2 + _weight_bytes(n, k, case) + (4 * n if case["bias"] else 0)
                + m * n_out * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    e, slots = case["experts"], case["tokens"] * case["k"]
    p = slots // case.get("share", 1)  # rows that have an expert here, about
    active = e * (1.0 - (1.0 - 1.0 / e) ** p)  # experts with a row, about
    if op == "grouped":
        n, k = case["n"], case["cols"]
        n_out = n // 2 if case["swiglu"] else n
        return {"bytes": p * k * 2 + active * _weight_bytes(n, k, case)
                + p * n_out * (2 if case["out"] == "bf16" else 4), "flops": 2 * p * n * k}
    if op == "layer":
        h, i = case["hidden"], case["inter"]
        return {"bytes": active * (_weight_bytes(2 * i, h, case) + _weight_bytes(h, i, case))
                + case["tokens"] * (4 * h + 8 * case["k"]), "flops": 6 * p * h * i}
    size = 2 if case["type"] == "bf16" else 4
    other = 2 if case.get("out", case["type"]) == "bf16" else 4
    many, few = p * case["hidden"], case["tokens"] * case["hidden"]
    if op == "dispatch":
        return {"bytes": size * (many + few) + 4 * (3 * slots + e), "flops": 4 * slots}
    if op == "dispatch_gradient":
        return {"bytes": size * (many + few) + 4 * slots, "flops": many}
    if op == "combine":
        more = size * few if case["shared"] else 0
        return {"bytes": size * many + other * few + more + 8 * slots, "flops": 2 * many}
    return {"bytes": 2 * size * many + other * few + 12 * slots, "flops": 3 * many}


# ---------------------------------------------------------- in 64 bits, apart --
def _weights64(w, ws, wz):
    """[n][k] in 64 bits, column by column of a group."""
    n, half = w.shape
    v = torch.empty(n, 2 * half, dtype=torch.float64, device=w.device)
    v[:, 0::2] = (w % 16).double()
    v[:, 1::2] = torch.div(w, 16, rounding_mode="floor").double()
    group = 2 * half // ws.shape[1]
    for c in range(ws.shape[1]):
        part = v[:, c * group:(c + 1) * group]
        part -= 8.0 if wz is None else wz[:, c:c + 1].double()
        part *= ws[:, c:c + 1].double()
    return v


def _swiglu64(y, swiglu):
    i = y.shape[1] // 2
    return y[:, :i] * torch.sigmoid(y[:, :i]) * y[:, i:] if swiglu else y


def _grouped64(x, offsets, w, swiglu):
    n = w[0].shape[1] // 2 if swiglu else w[0].shape[1]
    y = torch.zeros(x.shape[0], n, dtype=torch.float64, device=x.device)
    at = offsets.tolist()
    for e in range(len(at) - 1):
        if at[e] < at[e + 1]:
            one = [None if v is None else v[e] for v in w]
            y[at[e]:at[e + 1]] = _swiglu64(x[at[e]:at[e + 1]] @ _weights64(*one).t(), swiglu)
    return y


def _rows_of(idx, experts):
    """Slots by expert, one expert at a time, and the experts' first rows."""
    flat = idx.reshape(-1)
    parts = [(flat == e).nonzero()[:, 0] for e in range(experts)]
    counts = torch.tensor([0] + [len(q) for q in parts], device=idx.device)
    return torch.cat(parts), counts.cumsum(0)


def _sums64(rows, slots, weight, t, k, more):
    """Sum over each token's slots of weight * row."""
    y = torch.zeros(t, rows.shape[1], dtype=torch.float64, device=rows.device)
    for c in range(0, rows.shape[1], 256):  # a strip of columns at a time
        part = rows[:len(slots), c:c + 256].double() * weight[:, None]
        y[:, c:c + 256].index_add_(0, slots // k, part)
    return y if more is None else y + more.double()


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "w4":
        y = s["x"].double() @ _weights64(s["w"], s["ws"], s["wz"]).t()
        return _swiglu64(y if s["bias"] is None else y + s["bias"].double(), case["swiglu"])
    t, k = case["tokens"], case["k"]
    slots, offsets = _rows_of(s["idx"], case["experts"])
    if op == "grouped":
        return _grouped64(s["x"].double(), offsets, s["w"], case["swiglu"])
    gates = s["gates"].double().reshape(-1)[slots]
    if op == "layer":
        rows = s["x"].double()[slots // k]
        h = _grouped64(rows, offsets, s["w1"], True).to(torch.bfloat16).double()
        y = _grouped64(h, offsets, s["w2"], False).to(torch.bfloat16)
        return _sums64(y, slots, gates, t, k, None)
    if op == "dispatch":
        rows = torch.zeros(t * k, case["hidden"], dtype=torch.float64, device=DEV)
        rows[:len(slots)] = s["x"].double()[slots // k]
        return rows, None, None, None
    if op == "dispatch_gradient":
        return _sums64(s["rows"], slots, torch.ones_like(gates), t, k, None)
    if op == "combine":
        return _sums64(s["rows"], slots, gates, t, k, s["shared"])
    d = s["d_out"].double()
    d_rows = torch.zeros(t * k, case["hidden"], dtype=torch.float64, device=DEV)
    d_rows[:len(slots)] = d[slots // k] * gates[:, None]
    d_gates = torch.zeros(t * k, dtype=torch.float64, device=DEV)
    dots = [(d[q // k] * s["rows"][i:i + len(q)].double()).sum(dim=1)
            for i, q in zip(range(0, len(slots), 4096), slots.split(4096))]
    d_gates[slots] = torch.cat(dots) if dots else d_gates[:0]
    return d_rows, d_gates.view(t, k)
