"""The routed half of a layer, as cases to be timed and compared: the router's
choices sorted by expert ("sort"), tokens taken to that order and the experts'
results brought back with the route's weights ("combine", in training with both
directions' gradients), and the experts' products in 8-bit integers with a
scale for each token and each channel ("linear8", "gated8"), dense or by
expert.

With `own` false every case is computed in its plain form, elementary torch
operations in FP32 (FP64 where a value next to a rounding border decides an
integer) rounded once at the end; with `own` true by the library's kernels
(latent_projection_top_amd.experts).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _sort(name, rows, topk, total, first, experts):
    return {"name": name, "op": "sort", "rows": rows, "topk": topk, "total": total, "first": first,
            "experts": experts}


def _combine(name, rows, topk, total, first, experts, width, train, dtype, residual):
    return {"name": name, "op": "combine", "rows": rows, "topk": topk, "total": total, "first": first,
            "experts": experts, "width": width, "train": train, "dtype": dtype, "residual": residual}


def _linear8(name, rows, topk, total, first, experts, inputs, outputs, dtype, act, bias, residual):
    return {"name": name, "op": "linear8", "rows": rows, "topk": topk, "total": total, "first": first,
            "experts": experts, "inputs": inputs, "outputs": outputs, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual}


def _gated8(name, rows, topk, total, first, experts, inputs, inner, dtype, act):
    return {"name": name, "op": "gated8", "rows": rows, "topk": topk, "total": total, "first": first,
            "experts": experts, "inputs": inputs, "inner": inner, "dtype": dtype, "act": act}


def listed():
    return [
        # one decoded token's sixteen experts of all 896: latency
        _sort("sort-1x16", 1, 16, 896, 0, 896),
        # a prefill chunk on one of eight ranks, which holds 112 of the 896
        # experts: seven of eight choices are not its own
        _sort("sort-2047x16-share", 2047, 16, 896, 336, 112),
        # a training batch over every expert
        _sort("sort-16384x16", 16384, 16, 896, 0, 896),
        # a decode round's results brought back to the hidden width onto the
        # residual stream
        _combine("combine-serve-8x16x7168", 8, 16, 896, 0, 896, 7168, False, "bf16", True),
        # a small model's training step on one rank of two: half of the choices
        # elsewhere, rows of an odd width
        _combine("combine-train-333x6x1001-f16", 333, 6, 64, 32, 32, 1001, True, "f16", False),
        # a training batch's latent rows to every expert and back, with all
        # gradients: HBM bandwidth
        _combine("combine-train-4096x16x3584", 4096, 16, 896, 0, 896, 3584, True, "bf16", False),
        # a decode round through one dense matrix back to the hidden width:
        # weight streaming
        _linear8("linear8-8x2048x7168", 8, 0, 1, 0, 1, 2048, 7168, "bf16", "none", False, True),
        # sorted rows of a small model's experts, every size odd
        _linear8("linear8-333x6of40-1019x777-f16", 333, 6, 40, 0, 40, 1019, 777, "f16", "gelu", True, False),
        # a prefill chunk through a dense matrix, everything in the epilogue
        _linear8("linear8-2048x3584x7168", 2048, 0, 1, 0, 1, 3584, 7168, "bf16", "gelu_tanh", True, True),
        # a decode round on one of eight ranks: sixteen or so rows, most of
        # them alone with their expert
        _gated8("gated8-8x16of112-3584x2048", 8, 16, 896, 112, 112, 3584, 2048, "bf16", "silu"),
        # a prefill chunk there: some eighteen rows to an expert
        _gated8("gated8-1024x16of112-3584x2048", 1024, 16, 896, 112, 112, 3584, 2048, "bf16", "silu"),
        # a long batch there: some seventy rows to an expert, the largest
        _gated8("gated8-4096x16of112-3584x2048", 4096, 16, 896, 112, 112, 3584, 2048, "bf16", "silu"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over [lo, hi] by its logarithm; three of five are
    multiples of 16 as most models' are, the rest are as drawn."""
    n = _log_int(rng, lo, hi)
    return max(16, n // 16 * 16) if rng.random() < 0.6 else n


def _routing(rng, most_total, most_topk):
    """(topk, total, first, experts): all experts here, or one rank's share."""
    total = _log_int(rng, 2, most_total)
    topk = rng.randint(1, min(most_topk, total))
    ranks = rng.choice((1, 1, 2, 4, 8))
    experts = max(1, total // ranks)
    first = experts * rng.randrange(total // experts)
    return topk, total, first, experts


def draw(rng):
    op = rng.choice(("sort", "combine", "linear8", "gated8"))
    if op == "sort":
        topk, total, first, experts = _routing(rng, 896, 16)
        return {"op": op, "rows": _log_int(rng, 1, 16384), "topk": topk, "total": total, "first": first,
                "experts": experts}
    if op == "combine":
        topk, total, first, experts = _routing(rng, 896, 16)
        width = _size(rng, 64, 7168)
        rows = _log_int(rng, 1, 4096 * 16 * 3584 // (topk * width) if topk * width > 16 * 3584 else 4096)
        return {"op": op, "rows": rows, "topk": topk, "total": total, "first": first, "experts": experts,
                "width": width, "train": rng.random() < 0.5,
                "dtype": rng.choice(("bf16", "bf16", "f16", "f32")), "residual": rng.random() < 0.5}
    act = rng.choice(("silu", "gelu", "gelu_tanh", "relu"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    inputs = _size(rng, 128, 3584)
    if rng.random() < 0.5:
        topk, total, first, experts = 0, 1, 0, 1
        rows = _log_int(rng, 1, 2048)
    else:
        topk, total, first, experts = _routing(rng, 128, 16)
        rows = _log_int(rng, 1, 4096)
        if rows * topk > 32768:
            rows = 32768 // topk
    if op == "linear8":
        return {"op": op, "rows": rows, "topk": topk, "total": total, "first": first, "experts": experts,
                "inputs": inputs, "outputs": _size(rng, 128, 2048 if topk else 7168), "dtype": dtype,
                "act": rng.choice((act, "none")), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5}
    return {"op": op, "rows": rows, "topk": topk, "total": total, "first": first, "experts": experts,
            "inputs": inputs, "inner": _size(rng, 128, 1024 if topk else 4096), "dtype": dtype, "act": act}


# ------------------------------------------------------------------ inputs --

def _choices(case, gen):
    """ids [rows][topk] of distinct experts, as a router gives them: some
    experts are chosen several times as often as others."""
    dev = torch.device("cuda")
    liking = torch.randn(case["total"], generator=gen, device=dev) * 0.5
    logits = torch.randn(case["rows"], case["total"], generator=gen, device=dev) + liking
    return torch.topk(logits, case["topk"], dim=1).indices.to(torch.int32)


def _sorted(case, ids):
    """offsets, place and token of the choices sorted by expert, in int64:
    those of experts elsewhere come last, and `kept` is what remains."""
    rows, topk, n = case["rows"], case["topk"], case["experts"]
    local = ids.long().flatten() - case["first"]
    local = torch.where((local < 0) | (local >= n), torch.full_like(local, n), local)
    order = torch.argsort(local, stable=True)
    counts = torch.zeros(n + 1, dtype=torch.int64, device=ids.device).index_add_(
        0, local, torch.ones_like(local))
    offsets = torch.cat((torch.zeros_like(counts[:1]), torch.cumsum(counts, 0)[:n]))
    at = torch.arange(rows * topk, device=ids.device)
    place = torch.empty_like(at).scatter_(0, order, at)
    place = torch.where(local < n, place, torch.full_like(place, -1)).view(rows, topk)
    token = torch.where(at < offsets[n], order // topk, torch.full_like(at, -1))
    return offsets, place, token


def _inputs(case, seed):
    """The tensors of a case: activations N(0, 1) with one channel in a hundred
    ten times larger, as hidden rows have; 8-bit weights as those of normal
    matrices with a scale for each channel; route weights that sum to 1;
    incoming gradients N(0, 0.1^2)."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rows, topk = case["rows"], case["topk"]
    s = {}
    if case["op"] == "sort":
        s["ids"] = _choices(case, gen)
        return s
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    def activations(r, n):
        x = torch.randn(r, n, generator=gen, device=dev)
        big = torch.rand(n, generator=gen, device=dev) < 0.01
        return torch.where(big, x * 10.0, x).to(dt)

    if case["op"] == "combine":
        w, cap = case["width"], rows * topk
        _, place, _ = _sorted(case, _choices(case, gen))
        s["place"] = place.to(torch.int32)
        score = torch.rand(rows, topk, generator=gen, device=dev) + 0.25
        s["weights"] = score / score.sum(dim=1, keepdim=True)
        s["ys"] = normal(cap, w)
        s["residual"] = activations(rows, w) if case["residual"] else None
        if case["train"]:
            s["x"] = activations(rows, w)
            s["dy"] = normal(rows, w, scale=0.1)
            s["dxs"] = normal(cap, w, scale=0.1)
        return s

    k, e = case["inputs"], case["experts"]
    n = case["outputs"] if case["op"] == "linear8" else case["inner"]

    def weight():
        w = torch.empty(e, k, n, dtype=torch.int8, device=dev)
        for i in range(e):
            w[i] = (torch.randn(k, n, generator=gen, device=dev) * 35.0).round_().clamp_(-127, 127)
        return w, (torch.rand(e, n, generator=gen, device=dev) * 0.4 + 0.8) / (35.0 * k ** 0.5)

    sorted_rows = rows * topk if topk else rows
    if topk:
        offsets, _, token = _sorted(case, _choices(case, gen))
        s["offsets"] = offsets.to(torch.int32)
    if case["op"] == "gated8":
        s["x"] = activations(rows, k)
        if topk:
            s["token"] = token.to(torch.int32)
        s["w_gate"], s["scale_gate"] = weight()
        s["w_up"], s["scale_up"] = weight()
    else:
        s["x"] = activations(sorted_rows, k)
        s["w"], s["scale"] = weight()
        s["bias"] = normal(e, n, scale=0.5) if case["bias"] else None
        s["residual"] = activations(sorted_rows, n) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dev = torch.device("cuda")
    rows, topk = case["rows"], case["topk"]
    if not own:
        if s.get("offsets") is not None:  # which rows are whose, for the loop over experts
            s["bounds"] = s["offsets"].tolist()
        return s
    from latent_projection_top_amd import experts

    if case["op"] == "sort":
        s["plan"] = experts.SortPlan(rows, topk, case["experts"], first=case["first"])
        s["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device=dev)
        s["place"] = torch.empty(rows, topk, dtype=torch.int32, device=dev)
        # entries behind the last kept choice are left as they are
        s["token"] = torch.full((rows * topk,), -1, dtype=torch.int32, device=dev)
        s["workspace"] = s["plan"].new_workspace()
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "combine":
        w, cap = case["width"], rows * topk
        s["plan"] = experts.CombinePlan(rows, topk, w, dtype=dt)
        s["y"] = torch.empty(rows, w, dtype=dt, device=dev)
        if case["train"]:
            s.update(xs=torch.zeros(cap, w, dtype=dt, device=dev), dys=torch.zeros(cap, w, dtype=dt, device=dev),
                     dx=torch.empty(rows, w, dtype=dt, device=dev),
                     dweights=torch.empty(rows, topk, dtype=torch.float32, device=dev))
        return s
    sorted_rows = rows * topk if topk else rows
    if case["op"] == "linear8":
        s["plan"] = experts.Linear8Plan(sorted_rows, case["inputs"], case["outputs"], experts=case["experts"],
                                        activation=case["act"], dtype=dt)
        s["packed"] = experts.pack(s["plan"], s["w"])
        s["y"] = torch.zeros(sorted_rows, case["outputs"], dtype=dt, device=dev)
    else:
        s["plan"] = experts.Gated8Plan(sorted_rows, case["inputs"], case["inner"], experts=case["experts"],
                                       tokens=rows, activation=case["act"], dtype=dt)
        s["packed"] = experts.pack(s["plan"], s["w_gate"], s["w_up"])
        s["h"] = torch.zeros(sorted_rows, case["inner"], dtype=dt, device=dev)
    s["workspace"] = s["plan"].new_workspace()
    return s


# --------------------------------------------------------------------- run --

def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z * (z > 0).to(z.dtype)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _plain_sort(s, case):
    offsets, place, token = _sorted(case, s["ids"])
    return {"offsets": offsets.to(torch.int32), "place": place.to(torch.int32), "token": token.to(torch.int32)}


def _spread(case, values, place):
    """values [rows][topk][width] FP32 at their places; what no choice has is 0."""
    out = torch.zeros(case["rows"] * case["topk"] + 1, case["width"], dtype=torch.float32, device=values.device)
    out[place.reshape(-1)] = values.reshape(-1, case["width"])  # -1 is the spare last row
    return out[:-1]


def _collect(case, values, place, weights=None):
    """The sum over a row's choices of its values, FP32, choice by choice."""
    out = torch.zeros(case["rows"], case["width"], dtype=torch.float32, device=values.device)
    for j in range(case["topk"]):
        at = place[:, j]
        v = values[at.clamp(min=0)].float()
        if weights is not None:
            v = v * weights[:, j, None]
        out += torch.where((at >= 0)[:, None], v, torch.zeros_like(v))
    return out


def _plain_combine(s, case):
    dt = s["ys"].dtype
    place = s["place"].long()
    y = _collect(case, s["ys"], place, s["weights"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(dt)}
    if case["train"]:
        topk = case["topk"]
        dy = s["dy"].float()
        xs = _spread(case, s["x"].float()[:, None].expand(-1, topk, -1), place)
        dys = _spread(case, s["weights"][:, :, None] * dy[:, None], place)
        dw = torch.empty_like(s["weights"])
        for j in range(topk):
            at = place[:, j]
            dot = (dy * s["ys"][at.clamp(min=0)].float()).sum(dim=1)
            dw[:, j] = torch.where(at >= 0, dot, torch.zeros_like(dot))
        out.update(xs=xs.to(dt), dys=dys.to(dt), dweights=dw,
                   dx=_collect(case, s["dxs"], place).to(dt))
    return out


def _quantise(x):
    """Integers and the scale of each row; decided in FP64, since a row's
    values may lie next to a border between two integers."""
    x = x.double()
    most = x.abs().amax(dim=1, keepdim=True)
    q = torch.round(127.0 * x / torch.where(most > 0, most, torch.ones_like(most)))
    return q.float(), (most / 127.0).float()


def _segments(s, rows):
    if "bounds" not in s:
        return [(0, 0, rows)]
    b = s["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _plain_linear8(s, case):
    dt = s["x"].dtype
    q, sx = _quantise(s["x"])
    y = torch.zeros(q.shape[0], case["outputs"], dtype=torch.float32, device=q.device)
    for e, a, b in _segments(s, q.shape[0]):
        z = (q[a:b] @ s["w"][e].float()) * sx[a:b] * s["scale"][e]
        if s["bias"] is not None:
            z = z + s["bias"][e].float()
        z = _act(case["act"], z)
        y[a:b] = z if s["residual"] is None else z + s["residual"][a:b].float()
    return {"y": y.to(dt)}


def _plain_gated8(s, case):
    dt = s["x"].dtype
    q, sx = _quantise(s["x"])
    rows = case["rows"] * case["topk"] if case["topk"] else case["rows"]
    h = torch.zeros(rows, case["inner"], dtype=torch.float32, device=q.device)
    for e, a, b in _segments(s, rows):
        if case["topk"]:
            at = s["token"][a:b].long()
            qe, se = q[at], sx[at]
        else:
            qe, se = q, sx
        g = (qe @ s["w_gate"][e].float()) * se * s["scale_gate"][e]
        u = (qe @ s["w_up"][e].float()) * se * s["scale_up"][e]
        h[a:b] = _act(case["act"], g) * u
    return {"h": h.to(dt)}


def _own_sort(s, case):
    from latent_projection_top_amd import experts

    experts.sort(s["plan"], s["ids"], s["offsets"], s["place"], s["token"], s["workspace"])
    return {k: s[k] for k in ("offsets", "place", "token")}


def _own_combine(s, case):
    from latent_projection_top_amd import experts

    p = s["plan"]
    if not case["train"]:
        experts.combine(p, s["ys"], s["place"], s["weights"], s["y"], residual=s["residual"])
        return {"y": s["y"]}
    experts.gather(p, s["x"], s["place"], s["xs"])
    experts.combine(p, s["ys"], s["place"], s["weights"], s["y"], residual=s["residual"])
    experts.combine_backward(p, s["dy"], s["ys"], s["place"], s["weights"], s["dys"], s["dweights"])
    experts.gather_backward(p, s["dxs"], s["place"], s["dx"])
    return {k: s[k] for k in ("y", "xs", "dys", "dweights", "dx")}


def _own_linear8(s, case):
    from latent_projection_top_amd import experts

    experts.linear8(s["plan"], s["x"], s["packed"], s["scale"], s["y"], s["workspace"], offsets=s.get("offsets"),
                    bias=s["bias"], residual=s["residual"])
    return {"y": s["y"]}


def _own_gated8(s, case):
    from latent_projection_top_amd import experts

    experts.gated8(s["plan"], s["x"], s["packed"], s["scale_gate"], s["scale_up"], s["h"], s["workspace"],
                   offsets=s.get("offsets"), token=s.get("token"))
    return {"h": s["h"]}


_RUN = {"sort": (_plain_sort, _own_sort), "combine": (_plain_combine, _own_combine),
        "linear8": (_plain_linear8, _own_linear8), "gated8": (_plain_gated8, _own_gated8)}


def run(state):
    case = state["case"]
    return _RUN[case["op"]][1 if own else 0](state, case)


# ------------------------------------------------------------------- exact --

_EXACT_ACT = {
    "none": lambda z: z,
    "relu": torch.relu,
    "silu": torch.nn.functional.silu,
    "gelu": torch.nn.functional.gelu,
    "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
}


def _exact_sort(case, ids):
    """The definition, choice by choice on the host."""
    rows, topk, n, first = case["rows"], case["topk"], case["experts"], case["first"]
    of = [[] for _ in range(n)]
    for c, expert in enumerate(ids.flatten().tolist()):
        if first <= expert < first + n:
            of[expert - first].append(c)
    offsets, place, token = [0], [-1] * (rows * topk), [-1] * (rows * topk)
    p = 0
    for choices in of:
        for c in choices:
            place[c], token[p] = p, c // topk
            p += 1
        offsets.append(p)

    def tensor(v):
        return torch.tensor(v, dtype=torch.int32, device=ids.device)

    return {"offsets": tensor(offsets), "place": tensor(place).view(rows, topk), "token": tensor(token)}


def _exact_combine(case, s):
    """The forward definitions as products with a selection, differentiated by
    torch's autograd. Each row's choices are gathered in FP64, a slice of rows
    at a time."""
    rows, topk, width = case["rows"], case["topk"], case["width"]
    place = s["place"].long()
    on = (place >= 0).double()
    at = place.clamp(min=0)
    out = {"y": torch.empty(rows, width, dtype=torch.float64, device=place.device)}
    if case["train"]:
        spare = torch.zeros(2, rows * topk + 1, width, dtype=torch.float64, device=place.device)
        out["dweights"] = torch.empty(rows, topk, dtype=torch.float64, device=place.device)
        out["dx"] = torch.empty_like(out["y"])
    step = max(1, (1 << 26) // (topk * width))
    for r in range(0, rows, step):
        i = slice(r, min(rows, r + step))
        v = s["ys"][at[i]].double()
        w = s["weights"][i].double()
        if case["train"]:
            v.requires_grad_(True)
            w.requires_grad_(True)
        y = torch.matmul((w * on[i])[:, None], v)[:, 0]
        if s["residual"] is not None:
            y = y + s["residual"][i].double()
        out["y"][i] = y.detach()
        if not case["train"]:
            continue
        dv, dw = torch.autograd.grad(y, (v, w), s["dy"][i].double())
        out["dweights"][i] = dw
        x = s["x"][i].double().requires_grad_(True)
        xs = x[:, None] * on[i][:, :, None]
        out["dx"][i] = torch.autograd.grad(xs, x, s["dxs"][at[i]].double())[0]
        spare[0][place[i].flatten()] = xs.detach().reshape(-1, width)
        spare[1][place[i].flatten()] = dv.reshape(-1, width)
    if case["train"]:
        out["xs"], out["dys"] = spare[0][:-1], spare[1][:-1]
    return out


def _exact_product(case, s):
    """Rows of integers times integers, in FP64 (exact), with their scales."""
    rows, topk = case["rows"], case["topk"]
    x = s["x"].double()
    gated = case["op"] == "gated8"
    out_rows = rows * topk if topk else rows
    width = case["inner"] if gated else case["outputs"]
    out = torch.zeros(out_rows, width, dtype=torch.float64, device=x.device)
    most, _ = x.abs().max(dim=1)
    unit = torch.where(most > 0, most, torch.ones_like(most))[:, None]
    q = (x * 127.0 / unit).round()
    bounds = s["offsets"].tolist() if topk else [0, rows]
    act = _EXACT_ACT[case["act"]]
    for e in range(case["experts"]):
        i = slice(bounds[e], bounds[e + 1])
        if i.start == i.stop:
            continue
        of = s["token"][i].long() if gated and topk else i
        qe, step = q[of], most[of][:, None] / 127.0
        if gated:
            g = torch.mm(qe, s["w_gate"][e].double()) * step * s["scale_gate"][e].double()
            out[i] = act(g) * (torch.mm(qe, s["w_up"][e].double()) * step * s["scale_up"][e].double())
            continue
        z = torch.mm(qe, s["w"][e].double()) * step * s["scale"][e].double()
        if s["bias"] is not None:
            z = z + s["bias"][e].double()
        out[i] = act(z)
        if s["residual"] is not None:
            out[i] += s["residual"][i].double()
    return {"h" if gated else "y": out}


def exact(case, seed):
    """The same outputs in FP64 from the definitions; integers as they are."""
    s = _inputs(case, seed)
    if case["op"] == "sort":
        return _exact_sort(case, s["ids"])
    if case["op"] == "combine":
        out = _exact_combine(case, s)
        order = ("y", "xs", "dys", "dweights", "dx") if case["train"] else ("y",)
        return {k: out[k] for k in order}
    return _exact_product(case, s)


# -------------------------------------------------------------------- work --

def work(case):
    """Bytes of every input read once and every output written once, and the
    operations of the sums and products. A rank's share of the choices is
    taken as its share of the experts."""
    rows, topk = case["rows"], case["topk"]
    choices = rows * topk
    kept = choices * case["experts"] // case["total"] if topk else rows
    if case["op"] == "sort":
        return {"bytes": 4 * (2 * choices + kept + case["experts"] + 1), "flops": choices}
    e = DTYPES[case["dtype"]].itemsize
    if case["op"] == "combine":
        w = case["width"]
        once, many = rows * w * e, kept * w * e
        small = 8 * choices
        if not case["train"]:
            return {"bytes": many + once * (2 if case["residual"] else 1) + small, "flops": 2 * kept * w}
        return {"bytes": 4 * many + (4 + case["residual"]) * once + small + 4 * choices, "flops": 6 * kept * w}
    k, n = case["inputs"], case["outputs"] if case["op"] == "linear8" else case["inner"]
    planes = 2 if case["op"] == "gated8" else 1
    # experts that some row has, if rows were dealt evenly
    live = case["experts"] * (1.0 - (1.0 - 1.0 / case["experts"]) ** kept) if case["experts"] > 1 else 1.0
    rows_in = rows if planes == 2 else kept
    data = e * (rows_in * k + kept * n) + planes * live * n * (k + 4)
    if planes == 1:
        data += e * (live * n * case["bias"] + kept * n * case["residual"])
    return {"bytes": int(data), "flops": 2 * planes * kept * k * n}
