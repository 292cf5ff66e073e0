"""Cases of the layer's fused-epilogue and expert operators, their plain forms and their exact results.

Four operators, in the order in which a quantised transformer block calls them:

* ``tq_linear_act``      Y = act(Q4(X) Q4(R) s_x s_w + (X L1) L2 + bias) + residual, or, gated, the product of the
                         activated first half of the channels with the second half (plus residual);
* ``tq_expert_plan``     the rows of every expert: pairs (token, choice) sorted by expert, stably;
* ``tq_linear_experts``  the layer above with each sorted row taking the weights of its expert;
* ``tq_expert_combine``  Y[t] = residual[t] + sum_j weight[t, j] Z[pos[t, j]].

With ``own`` false, ``run`` computes them with elementary torch operations in fp32 (the quantiser's division in fp64,
so that no code next to a rounding border differs); with ``own`` true it calls the library.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def listed():
    return [
        # gate and up of an 8B MLP with its SiLU product, one token: the decode step, bound by the weights
        dict(name="act gate/up 1 token", op="act", n=1, d=4096, m=28672, r=64, x="bf16", y="bf16", act="silu", gated=True,
             bias=False, res="none"),
        # a small biased GELU layer in fp32 with a few tokens and odd sizes: latency alone
        dict(name="act small fp32 odd", op="act", n=7, d=512, m=1001, r=16, x="f32", y="f32", act="gelu", gated=False,
             bias=True, res="f32"),
        # an attention output projection over a prompt, added to the residual stream
        dict(name="act proj 4096 residual", op="act", n=4096, d=4096, m=4096, r=32, x="bf16", y="bf16", act="none", gated=False,
             bias=False, res="bf16"),
        # gate and up of the 8B MLP over a prompt of ragged length
        dict(name="act gate/up 2047", op="act", n=2047, d=4096, m=28672, r=64, x="bf16", y="bf16", act="silu", gated=True,
             bias=False, res="none"),
        # the routing of a decode batch: one small launch
        dict(name="plan 16 tokens", op="plan", n=16, topk=8, E=128, drop=0.0, ids="i64"),
        # the routing of a long prefill batch with padding tokens dropped
        dict(name="plan 32768 tokens", op="plan", n=32768, topk=8, E=256, drop=0.05, ids="i64"),
        # eight large experts, four sequences decoding: gate and up, bound by the weights of the active experts
        dict(name="experts gate/up 4 tokens", op="experts", n=4, topk=2, E=8, d=4096, m=28672, r=64, gather=True, drop=0.0,
             x="bf16", y="bf16", act="silu", gated=True, bias=False),
        # many small experts, a decode batch: the down product on rows in sorted order
        dict(name="experts down 24 tokens", op="experts", n=24, topk=6, E=64, d=1408, m=2048, r=32, gather=False, drop=0.0,
             x="bf16", y="bf16", act="none", gated=False, bias=False),
        # many small experts with biases, a ragged prefill chunk whose padding is dropped
        dict(name="experts gate/up 1111 tokens", op="experts", n=1111, topk=8, E=128, d=2048, m=1536, r=32, gather=True, drop=0.1,
             x="bf16", y="bf16", act="silu", gated=True, bias=True),
        # eight large experts, a prefill batch: the largest product
        dict(name="experts gate/up 4096 tokens", op="experts", n=4096, topk=2, E=8, d=4096, m=28672, r=64, gather=True, drop=0.0,
             x="bf16", y="bf16", act="silu", gated=True, bias=False),
        # the weighted sum of a decode batch's expert outputs onto the residual stream
        dict(name="combine 4 tokens", op="combine", n=4, topk=2, m=4096, drop=0.0, z="bf16", y="bf16", res="bf16", w="f32"),
        # the same for a prefill batch of many small experts
        dict(name="combine 4095 tokens", op="combine", n=4095, topk=8, m=4096, drop=0.05, z="bf16", y="bf16", res="bf16", w="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the same ranges: one to some thousands of tokens, d from 64 to 8192, odd channel counts, both types."""
    op = rng.choice(["act", "act", "experts", "experts", "plan", "combine"])
    if op == "plan":
        E = _log(rng, 2, 512)
        return dict(op="plan", n=_log(rng, 1, 20000), topk=rng.randint(1, min(8, E)), E=E, drop=rng.choice([0.0, 0.07]),
                    ids=rng.choice(["i32", "i64"]))
    if op == "combine":
        return dict(op="combine", n=_log(rng, 1, 4000), topk=rng.randint(1, 8), m=_log(rng, 64, 4096), drop=rng.choice([0.0, 0.2]),
                    z=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "f32"]), res=rng.choice(["none", "bf16", "f32"]),
                    w=rng.choice(["f32", "bf16"]))
    c = dict(op=op, d=32 * _log(rng, 2, 256), r=rng.choice([0, 8, 16, 32, 48, 64, 100, 128]), x=rng.choice(["bf16", "bf16", "f32"]),
             y=rng.choice(["bf16", "bf16", "f32"]), act=rng.choice(sorted(ACT)), gated=rng.random() < 0.4, bias=rng.random() < 0.5)
    if op == "act":
        c.update(n=_log(rng, 1, 2500), m=_log(rng, 48, 9000), res=rng.choice(["none", "bf16", "f32"]))
    else:
        E = _log(rng, 2, 96)
        c.update(E=E, topk=rng.randint(1, min(8, E)), n=_log(rng, 1, 900), m=_log(rng, 48, 2800), gather=rng.random() < 0.6,
                 drop=rng.choice([0.0, 0.1]))
        c["d"] = min(c["d"], 4096)
    c["m"] += c["m"] % 2 if c["gated"] else 0
    return c


# --------------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------------
def _layer(case, g, E):
    """Packed weights as tq_pack_weight and tq_pack_lowrank lay them out: E stacked layers of m channels."""
    d, m, r = case["d"], case["m"], case["r"]
    dev = "cuda"
    w_codes = torch.empty((E * m, d // 2), dtype=torch.uint8, device=dev)
    w_codes.random_(0, 256, generator=g)
    s_w = (0.5 + torch.rand(E * m, device=dev, generator=g)) * (0.25 / math.sqrt(d))
    blobs, rp = None, 0
    if r > 0:
        rp = 32
        while rp < r:
            rp *= 2
        l1 = torch.zeros((E, rp, d), device=dev)
        l1[:, :r] = torch.randn((E, r, d), device=dev, generator=g) / math.sqrt(d)
        l2 = torch.zeros((E, m, rp), device=dev)
        l2[:, :, :r] = torch.randn((E, m, r), device=dev, generator=g) * (0.5 / math.sqrt(r))
        blobs = torch.cat([l1.reshape(E, -1), l2.reshape(E, -1)], dim=1).bfloat16().contiguous()
    return dict(w_codes=w_codes, s_w=s_w, lowrank=blobs, rp=rp,
                bias=torch.randn(E * m, device=dev, generator=g) * 0.5 if case["bias"] else None)


def _act_rows(n, d, dt, g):
    """Activations with a few large channels, as they reach a layer behind a norm."""
    x = torch.randn((n, d), device="cuda", generator=g)
    gain = torch.ones(d, device="cuda")
    gain[torch.randperm(d, device="cuda", generator=g)[: max(1, d // 1000)]] = 10.0
    return (x * gain).to(DT[dt])


def _route(case, g):
    """topk distinct experts of every token, some experts far more popular than others; -1 in a dropped token's row."""
    n, k, E = case["n"], case["topk"], case["E"]
    score = torch.randn((n, E), device="cuda", generator=g) + 0.7 * torch.randn(E, device="cuda", generator=g)
    ids = score.topk(k, dim=1).indices
    if case["drop"] > 0:
        ids = torch.where(torch.rand((n, 1), device="cuda", generator=g) < case["drop"], -1, ids)
    return ids


def _sorted_rows(ids, E):
    """(offsets, order, pos) of the documented plan, entries behind the last kept pair zero."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    by = torch.sort(key, stable=True)
    order = torch.where(by.values < E, by.indices, 0).int()
    pos = torch.empty_like(flat, dtype=torch.int32)
    pos[by.indices] = torch.where(by.values < E, torch.arange(flat.numel(), device=flat.device), -1).int()
    offsets = (by.values[None, :] < torch.arange(E + 1, device=flat.device)[:, None]).sum(1).int()
    return offsets, order, pos.reshape(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "plan":
        s["ids"] = _route(case, g).to(torch.int64 if case["ids"] == "i64" else torch.int32).contiguous()
        P = case["n"] * case["topk"]
        if own:
            import rank_augmented_quantized_amd as tq
            s["ws"] = tq.expert_plan_workspace(case["n"], case["topk"], case["E"], "cuda")
        s["out"] = (torch.zeros(case["E"] + 1, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda"),
                    torch.zeros((case["n"], case["topk"]), dtype=torch.int32, device="cuda"))
    elif case["op"] == "combine":
        n, k, m = case["n"], case["topk"], case["m"]
        ids = torch.rand((n, k), device="cuda", generator=g)
        pos = ids.reshape(-1).argsort().argsort().int().reshape(n, k)
        if case["drop"] > 0:
            pos = torch.where(torch.rand((n, k), device="cuda", generator=g) < case["drop"], -1, pos)
        s["pos"] = pos.contiguous()
        s["weights"] = torch.softmax(torch.randn((n, k), device="cuda", generator=g), dim=1).to(DT[case["w"]])
        s["Z"] = torch.randn((n * k, m), device="cuda", generator=g).to(DT[case["z"]])
        s["res"] = None if case["res"] == "none" else torch.randn((n, m), device="cuda", generator=g).to(DT[case["res"]])
        s["Y"] = torch.empty((n, m), dtype=DT[case["y"]], device="cuda")
    else:
        n, d, m, r = case["n"], case["d"], case["m"], case["r"]
        mo = m // 2 if case["gated"] else m
        if case["op"] == "act":
            s.update(_layer(case, g, 1))
            s["X"] = _act_rows(n, d, case["x"], g)
            s["res"] = None if case["res"] == "none" else torch.randn((n, mo), device="cuda", generator=g).to(DT[case["res"]])
            s["Y"] = torch.empty((n, mo), dtype=DT[case["y"]], device="cuda")
        else:
            E, k = case["E"], case["topk"]
            s.update(_layer(case, g, E))
            ids = _route(case, g)
            s["offsets"], s["order"], s["pos"] = _sorted_rows(ids, E)
            s["X"] = _act_rows(n if case["gather"] else n * k, d, case["x"], g)
            s["Y"] = torch.zeros((n * k, mo), dtype=DT[case["y"]], device="cuda")
            counts = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
            # what the plain form's batch of padded segments needs to know on the host
            s["cap"] = max(counts + [1])
            s["active"] = torch.tensor([e for e, c in enumerate(counts) if c] or [0], device="cuda")
        if own:
            import rank_augmented_quantized_amd as tq
            if case["op"] == "act":
                s["ws"] = tq.linear_act_workspace(n, d, m, r, "cuda")
            else:
                k = case["topk"] if case["gather"] else 1
                s["ws"] = tq.linear_experts_workspace(s["X"].shape[0], k, d, m, r, case["E"], "cuda")
    return s


# --------------------------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------------------------
def _codes(packed):
    """Two's-complement nibbles, the even index low, to fp32 values."""
    lo = (packed & 15).to(torch.int8)
    hi = (packed >> 4).to(torch.int8)
    both = torch.stack([lo, hi], dim=-1).flatten(-2)
    return torch.where(both > 7, both - 16, both).float()


def _quantise(x):
    """Per row s = fl32(max|x| / 7) and the codes rne(fl32(x / s)), the divisions in fp64 and rounded to fp32."""
    amax = x.float().abs().amax(-1, keepdim=True)
    s = (amax.double() / 7).float()
    q = (x.double() / torch.where(s > 0, s, 1).double()).float().round().clamp(-8, 7)
    return torch.where(s > 0, q, 0), s


def _activate(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _finish(v, case):
    """The epilogue after the bias: activation, or the activated first half times the second."""
    if not case["gated"]:
        return _activate(v, case["act"])
    h = case["m"] // 2
    return _activate(v[..., :h], case["act"]) * v[..., h:]


def _plain_act(s):
    case = s["case"]
    d, m, rp = case["d"], case["m"], s["rp"]
    q, sx = _quantise(s["X"])
    v = (q @ _codes(s["w_codes"]).T) * (sx * s["s_w"])
    if rp:
        blob = s["lowrank"][0]
        l1, l2 = blob[: rp * d].reshape(rp, d).float(), blob[rp * d:].reshape(m, rp).float()
        v = v + (s["X"].bfloat16().float() @ l1.T) @ l2.T
    if s["bias"] is not None:
        v = v + s["bias"]
    y = _finish(v, case)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(DT[case["y"]])


def _plain_plan(s):
    return _sorted_rows(s["ids"], s["case"]["E"])


def _plain_experts(s):
    """Every active expert's rows padded to the longest segment, one batched product over the active experts."""
    case = s["case"]
    E, m, d, rp, cap, active = case["E"], case["m"], case["d"], s["rp"], s["cap"], s["active"]
    start = s["offsets"][active].long()
    count = s["offsets"][active + 1].long() - start
    row = start[:, None] + torch.arange(cap, device="cuda")
    kept = torch.arange(cap, device="cuda") < count[:, None]
    row = torch.where(kept, row, 0)
    src = s["order"].long()[row] // case["topk"] if case["gather"] else row
    q, sx = _quantise(s["X"])
    w = _codes(s["w_codes"].reshape(E, m, d // 2)[active])
    sw = s["s_w"].reshape(E, 1, m)[active]
    v = torch.bmm(q[src], w.transpose(1, 2).contiguous()) * (sx[src] * sw)
    if rp:
        blob = s["lowrank"][active]
        l1 = blob[:, : rp * d].reshape(-1, rp, d).float().transpose(1, 2).contiguous()
        l2 = blob[:, rp * d:].reshape(-1, m, rp).float().transpose(1, 2).contiguous()
        v = v + torch.bmm(torch.bmm(s["X"].bfloat16().float()[src], l1), l2)
    if s["bias"] is not None:
        v = v + s["bias"].reshape(E, 1, m)[active]
    y = _finish(v, case).to(DT[case["y"]])
    out = torch.zeros((s["Y"].shape[0] + 1, y.shape[-1]), dtype=y.dtype, device="cuda")
    out[torch.where(kept, row, s["Y"].shape[0])] = y
    return out[:-1]


def _plain_combine(s):
    case = s["case"]
    keep = s["pos"] >= 0
    z = s["Z"].float()[torch.where(keep, s["pos"], 0).long()]
    y = (torch.where(keep, s["weights"].float(), 0)[..., None] * z).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(DT[case["y"]])


def _own(s):
    import rank_augmented_quantized_amd as tq

    case = s["case"]
    if case["op"] == "plan":
        offsets, order, pos = s["out"]
        return tq.tq_expert_plan(s["ids"], case["E"], offsets=offsets, order=order, pos=pos, ws=s["ws"])
    if case["op"] == "combine":
        return tq.tq_expert_combine(s["Z"], s["pos"], s["weights"], residual=s["res"], Y=s["Y"])
    if case["op"] == "act":
        return tq.tq_linear_act(s["X"], s["w_codes"], s["s_w"], s["lowrank"], case["m"], case["r"], bias=s["bias"],
                                act=ACT[case["act"]], gated=case["gated"], residual=s["res"], Y=s["Y"], ws=s["ws"])
    return tq.tq_linear_experts(s["X"], s["w_codes"], s["s_w"], s["lowrank"], case["m"], case["r"], s["offsets"],
                                order=s["order"] if case["gather"] else None, topk=case["topk"] if case["gather"] else 1,
                                bias=s["bias"], act=ACT[case["act"]], gated=case["gated"], Y=s["Y"], ws=s["ws"])


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "combine": _plain_combine, "act": _plain_act, "experts": _plain_experts}[state["case"]["op"]](state)


def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0}
    if case["op"] == "plan":
        P = case["n"] * case["topk"]
        return {"bytes": P * (8 if case["ids"] == "i64" else 4) + 8 * P + 4 * (case["E"] + 1), "flops": 0}
    if case["op"] == "combine":
        n, k, m = case["n"], case["topk"], case["m"]
        return {"bytes": n * k * m * size[case["z"]] * (1 - case["drop"]) + n * m * (size[case["y"]] + size[case["res"]])
                + n * k * (4 + size[case["w"]]), "flops": 2 * n * k * m}
    n, d, m, r = case["n"], case["d"], case["m"], case["r"]
    mo = m // 2 if case["gated"] else m
    layer = m * d / 2 + 4 * m + 2 * r * (d + m) + (4 * m if case["bias"] else 0)
    if case["op"] == "act":
        rows, layers, extra, xrows = n, 1, n * mo * size[case["res"]], n
    else:
        rows = n * case["topk"] * (1 - case["drop"])
        # an expert is read if a token chose it; tokens choose topk of E experts
        layers = case["E"] * (1 - (1 - case["topk"] / case["E"]) ** n)
        extra, xrows = 8 * n * case["topk"], n if case["gather"] else rows
    return {"bytes": layers * layer + xrows * d * size[case["x"]] + rows * mo * size[case["y"]] + extra,
            "flops": 2 * rows * (d * m + r * (d + m))}


# --------------------------------------------------------------------------------------------------------------------
# exact results: the definitions in fp64, row by row of the sorted pairs
# --------------------------------------------------------------------------------------------------------------------
def _exact_rows(X, w_bytes, s_w, l1t, l2t, bias, case):
    """fp64 rows of one layer: exact code sums, unrounded low-rank branch, the activation's definition."""
    x = X.double()
    sx = (x.abs().max(dim=1).values / 7.0).to(torch.float32).double()
    ratio = (x / torch.where(sx == 0, torch.ones_like(sx), sx)[:, None]).to(torch.float32).double()
    cx = torch.clamp(torch.round(ratio), -8, 7) * (sx > 0)[:, None]
    w = torch.empty((w_bytes.shape[0], 2 * w_bytes.shape[1]), dtype=torch.float64, device=w_bytes.device)
    w[:, 0::2] = torch.remainder(w_bytes.to(torch.int16), 16).double()
    w[:, 1::2] = torch.div(w_bytes.to(torch.int16), 16, rounding_mode="floor").double()
    w -= 16.0 * (w >= 8)
    v = (cx @ w.t()) * sx[:, None] * s_w.double()[None, :]
    if l1t is not None:
        v += (X.to(torch.bfloat16).double() @ l1t.double().t()) @ l2t.double().t()
    if bias is not None:
        v += bias.double()[None, :]
    a = v[:, : v.shape[1] // 2] if case["gated"] else v
    kind = case["act"]
    if kind == "relu":
        a = torch.where(a > 0, a, torch.zeros_like(a))
    elif kind == "silu":
        a = a * torch.special.expit(a)
    elif kind == "gelu":
        a = 0.5 * a * torch.special.erfc(-a * math.sqrt(0.5))
    elif kind == "gelu_tanh":
        a = a * torch.special.expit(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
    return a * v[:, v.shape[1] // 2:] if case["gated"] else a


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "combine":
        Z, n, k = s["Z"].double(), case["n"], case["topk"]
        y = s["res"].double() if s["res"] is not None else torch.zeros((n, case["m"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            p = s["pos"][:, j].long()
            on = (p >= 0).nonzero()[:, 0]
            y[on] += s["weights"][on, j].double()[:, None] * Z[p[on]]
        return y
    d, m, rp = case["d"], case["m"], s["rp"]

    def factors(e):
        if not rp:
            return None, None
        b = s["lowrank"][e]
        return b[: rp * d].view(rp, d), b[rp * d:].view(m, rp)

    if case["op"] == "act":
        y = _exact_rows(s["X"], s["w_codes"], s["s_w"], *factors(0), s["bias"], case)
        return y + s["res"].double() if s["res"] is not None else y
    out = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda")
    off = s["offsets"].tolist()
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x = s["X"][(s["order"][a:b] // case["topk"]).long()] if case["gather"] else s["X"][a:b]
        c = slice(e * m, (e + 1) * m)
        out[a:b] = _exact_rows(x, s["w_codes"][c], s["s_w"][c], *factors(e), s["bias"][c] if s["bias"] is not None else None, case)
    return out
