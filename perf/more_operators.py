"""Cases, inputs and plain forms of the 8-bit integer path, for timing and checking it.

Three operators carry a layer whose checkpoint holds 8-bit integer weights with
one scale for each output channel, and whose activations are quantised per token
while it runs:

``dispatch``  layout and dispatch with the rows quantised as they are written: for each
              token s = amax/127 in fp32, codes RNE(x/s), one scale a receive row
``gated``     both input projections of each expert, the SiLU and the product, and the
              result quantised again:  h = silu(x Wg^T) * (x Wu^T), s = amax/127 over h's row
``down``      each expert's output product:  y = h W2^T

A value of a row is code * row scale, one of a weight code * channel scale. Rows are
in receive order (expert-contiguous segments named by expert_offset); weights are
w13 [E, 2F, H] (gate rows, then up rows) with scales [E, 2F], and w2 [E, H, F] with
scales [E, H].

A case is a dict of plain values; prepare() draws its inputs on the GPU, run()
makes one pass (the plain form in 32 bits, or the library's kernels when ``own``
is true), exact() gives the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

INT8_MAX = 127.0


# ---- cases ----------------------------------------------------------------
def listed():
    return [
        # one token of a small layer: launch latency is all there is
        dict(name="dispatch one token", op="dispatch", P=1, E=8, T=1, k=2, H=1024,
             routing="uniform", masked=0.0, cap=0),
        # the decode workload's batch
        dict(name="dispatch decode", op="dispatch", P=8, E=256, T=1024, k=8, H=7168,
             routing="uniform", masked=0.0, cap=0),
        # odd sizes, padded slots, hot experts cut at a capacity
        dict(name="dispatch ragged", op="dispatch", P=4, E=32, T=1332, k=3, H=2064,
             routing="zipf", masked=0.05, cap=200),
        # a prefill step of the headline layer
        dict(name="dispatch prefill", op="dispatch", P=32, E=256, T=32768, k=8, H=7168,
             routing="uniform", masked=0.0, cap=0),
        # one token of a small layer
        dict(name="gated one token", op="gated", E=8, T=1, k=2, H=1024, F=512, routing="uniform"),
        # the decode workload's batch: every expert's weights stream once
        dict(name="gated decode", op="gated", E=256, T=1024, k=8, H=7168, F=2048,
             routing="uniform"),
        # an odd decode batch with sizes that no tile divides
        dict(name="gated ragged", op="gated", E=32, T=333, k=4, H=4112, F=1008, routing="uniform"),
        # the uniform workload, 512 rows an expert: arithmetic bound
        dict(name="gated uniform", op="gated", E=64, T=16384, k=2, H=7168, F=2048,
             routing="uniform"),
        # the skewed workload: hot experts
        dict(name="gated skewed", op="gated", E=8, T=32768, k=2, H=4096, F=1408, routing="zipf"),
        # one token of the decode workload: eight experts of one row each
        dict(name="down one token", op="down", E=256, T=1, k=8, H=7168, F=2048,
             routing="uniform"),
        # one dense block (a single expert that every token takes)
        dict(name="down dense", op="down", E=1, T=4096, k=1, H=7168, F=2048, routing="uniform"),
        # a prefill chunk over the decode workload's experts
        dict(name="down prefill", op="down", E=256, T=16384, k=8, H=7168, F=2048,
             routing="uniform"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges: sizes by their logarithm, odd ones among them."""
    op = rng.choice(["dispatch", "gated", "down"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    E = _log_int(rng, 1, 256)
    c = dict(op=op, E=E, T=_log_int(rng, 1, 32768), k=rng.randint(1, min(8, E)),
             routing=rng.choice(["uniform", "zipf"]), H=16 * _log_int(rng, 16, 448))
    if op == "dispatch":
        c["P"] = rng.choice([p for p in (1, 2, 4, 8, 16, 32) if E % p == 0])
        c["T"] = max(1, c["T"] // c["P"]) * c["P"]
        c["masked"] = rng.choice([0.0, 0.05, 0.3])
        c["cap"] = rng.choice([0, 0, max(1, c["T"] * c["k"] // E)])
    else:
        c["F"] = 16 * _log_int(rng, 8, 176)
    while _cost(c) > most:
        if c["T"] > 64:
            c["T"] = c["T"] // 2 // c.get("P", 1) * c.get("P", 1)
        else:
            c["E"] = max(c.get("P", 1), c["E"] // 2 // c.get("P", 1) * c.get("P", 1))
            c["k"] = min(c["k"], c["E"])
    return c


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 7e12, w["flops"] / 2e15)


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    E, T, k, H = case["E"], case["T"], case["k"], case["H"]
    rows = T * k
    if case["op"] == "dispatch":
        kept = rows - _masked(case)
        if case["cap"] and case["routing"] == "uniform":
            kept = min(kept, E * case["cap"])
        # x, ids and weights in; codes, scale and 20 bytes of metadata a row, inv out
        return {"bytes": T * H * 2 + rows * 12 + kept * (H + 24), "flops": T * H * 3}
    F = case["F"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts with a row, at uniform routing
    if case["op"] == "gated":
        return {"bytes": used * 2 * F * (H + 4) + rows * (H + F + 8), "flops": 4 * rows * H * F}
    return {"bytes": used * H * (F + 4) + rows * (F + 4 + 2 * H), "flops": 2 * rows * H * F}


def _masked(case):
    """Padded slots of a dispatch case."""
    return int(case["T"] * case["k"] * case["masked"])


# ---- inputs ---------------------------------------------------------------
def _route(case, gen):
    """[T, k] distinct experts of each token: uniform, or Zipf(1.2) without replacement."""
    E, T, k = case["E"], case["T"], case["k"]
    u = torch.rand(T, E, generator=gen, device="cuda").clamp_min_(1e-20)
    keys = -torch.log(-torch.log(u))
    if case["routing"] == "zipf":
        keys -= 1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return keys.topk(k, dim=1).indices.to(torch.int32).contiguous()


def _normal(gen, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def _quantised(v):
    """int8 codes and fp32 scales amax/127 of each row of a matrix, of 32-bit values."""
    amax = v.abs().amax(-1)
    s = amax / torch.full_like(amax, INT8_MAX)  # a quotient: by a number it would be a product
    q = torch.where(s[..., None] > 0, v / s[..., None], 0.0)
    return torch.round(q).to(torch.int8), s


def _quantised_rows(gen, rows, n, gated=False):
    """Activations: normal values, or silu(g) u of normal g and u."""
    codes = torch.empty(rows, n, dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    for lo in range(0, rows, 65536):  # bounds the 32-bit copy
        v = torch.empty(min(65536, rows - lo), n, device="cuda").normal_(generator=gen)
        if gated:
            v = _silu32(v) * torch.empty_like(v).normal_(generator=gen)
        codes[lo:lo + 65536], scale[lo:lo + 65536] = _quantised(v)
    return codes, scale


def _quantised_weights(gen, E, n, m):
    """Normal weights [E, n, m] of deviation m^-1/2, channels of unlike size."""
    codes = torch.empty(E, n, m, dtype=torch.int8, device="cuda")
    scale = torch.empty(E, n, device="cuda")
    step = max(1, (1 << 28) // (n * m))
    for lo in range(0, E, step):
        e = min(step, E - lo)
        v = torch.empty(e, n, m, device="cuda").normal_(0.0, m ** -0.5, generator=gen)
        v *= 0.5 + torch.rand(e, n, 1, generator=gen, device="cuda")
        codes[lo:lo + e], scale[lo:lo + e] = _quantised(v)
    return codes, scale


def _plan(counts, rows):
    """Segments of the rows by expert, for the plain form: the experts that have rows, and
    either a padded row index (one batched product) or, where padding would cost more than
    half as much again, one product for each of them."""
    offset = [0]
    for n in counts:
        offset.append(offset[-1] + n)
    active = [e for e, n in enumerate(counts) if n]
    plan = {"rows": rows, "spans": [(e, offset[e], offset[e + 1]) for e in active], "pad": None}
    widest = max(counts)
    if active and len(active) * widest <= rows * 1.5 + 2048:
        n = torch.tensor([counts[e] for e in active], device="cuda")
        first = torch.tensor([offset[e] for e in active], device="cuda")
        at = torch.arange(widest, device="cuda")
        valid = at[None, :] < n[:, None]
        plan["active"] = torch.tensor(active, device="cuda")
        plan["pad"] = torch.where(valid, first[:, None] + at[None, :], rows)  # row `rows` is zero
        plan["unpad"] = valid.flatten().nonzero().flatten()
    return plan


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    E, T, k, H = case["E"], case["T"], case["k"], case["H"]
    ids = _route(case, gen)
    if case["op"] == "dispatch":
        return _prepare_dispatch(case, gen, ids)
    F, rows = case["F"], T * k
    count = torch.bincount(ids.flatten(), minlength=E)
    s = {"op": case["op"], "case": dict(case), "plan": _plan(count.tolist(), rows),
         "offset": torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)}
    if case["op"] == "gated":
        s["x"], s["xs"] = _quantised_rows(gen, rows, H)
        s["w13"], s["w13s"] = _quantised_weights(gen, E, 2 * F, H)
    else:
        s["hid"], s["hids"] = _quantised_rows(gen, rows, F, gated=True)
        s["w2"], s["w2s"] = _quantised_weights(gen, E, H, F)
    if own:
        import combine_top_histogram_gb300 as moe
        s["moe"] = moe
        s["h"] = moe.moe_expert_create(moe.make_expert_config(E, H, F, rows, moe.MOE_INT8))
        if case["op"] == "gated":
            s["out"] = torch.empty(rows, F, dtype=torch.int8, device="cuda")
            s["outs"] = torch.empty(rows, device="cuda")
        else:
            s["out"] = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_dispatch(case, gen, ids):
    P, E, T, k, H = case["P"], case["E"], case["T"], case["k"], case["H"]
    padded = torch.randperm(T * k, generator=gen, device="cuda")[:_masked(case)]
    ids.view(-1)[padded] = -1
    w = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), 1)
    x = _normal(gen, T, H)
    x *= 0.25 + torch.rand(T, 1, generator=gen, device="cuda").to(x.dtype)  # tokens of unlike size
    # rows of the receive buffers: those that no assignment takes stay as they are, zero here
    s = {"op": "dispatch", "case": dict(case), "ids": ids, "w": w, "x": x,
         "rows": min(T * k, E * case["cap"] if case["cap"] else T * k)}
    if own:
        import combine_top_histogram_gb300 as moe
        s["layer"] = moe.MoeLayer(P, T // P, E, k, H, moe.MOE_INT8, case["cap"])
        s["layer"].poison(0)
        s["inv"] = s["layer"].layout_view()["inv"]
    return s


# ---- one pass -------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    if s["op"] == "dispatch":
        layer = s["layer"]
        layer.layout(s["ids"])
        layer.dispatch(s["x"], s["w"])
        return {"recv_x": layer.recv_x, "recv_scale": layer.recv_scale,
                "inv": s["inv"], "weight": layer.meta["weight"],
                "src_token": layer.meta["src_token"], "slot": layer.meta["slot"]}
    moe = s["moe"]
    if s["op"] == "gated":
        moe.moe_expert_gated(s["h"], s["offset"], s["x"], s["xs"], s["w13"], s["w13s"], s["out"],
                             s["outs"])
        return {"hid": s["out"].to(torch.bfloat16), "hid_scale": s["outs"]}  # codes, as numbers
    moe.moe_expert_down(s["h"], s["offset"], s["hid"], s["hids"], s["w2"], s["w2s"], s["out"])
    return {"y": s["out"]}


def _silu32(g):
    return g / (1.0 + torch.exp(-g))


def _product(p, a, w, ws):
    """Each row of a (32 bits) times its expert's matrix w[e]^T (codes times channel scales)."""
    if p["pad"] is not None:
        v = w[p["active"]].float().mul_(ws[p["active"]][..., None])
        padded = torch.cat([a, a.new_zeros(1, a.shape[1])])[p["pad"]]
        out = torch.bmm(padded, v.transpose(1, 2))
        return out.reshape(-1, out.shape[2])[p["unpad"]]
    out = torch.empty(p["rows"], w.shape[1], device="cuda")
    for e, lo, hi in p["spans"]:
        out[lo:hi] = a[lo:hi] @ (w[e].float() * ws[e][:, None]).T
    return out


def _run_plain(s):
    c = s["case"]
    if s["op"] == "dispatch":
        T, k, E, n = c["T"], c["k"], c["E"], s["rows"]
        # receive order: (expert, source rank, token, slot); padded slots have no row
        flat = s["ids"].flatten().long()
        key = torch.where(flat < 0, E, flat)
        order = torch.argsort(key, stable=True)
        sorted_key = key[order]
        first = torch.searchsorted(sorted_key, torch.arange(E + 1, device="cuda"))
        place = torch.arange(T * k, device="cuda") - first[sorted_key]  # within the expert
        kept = sorted_key < E
        if c["cap"]:
            kept &= place < c["cap"]
        row = torch.where(kept, torch.cumsum(kept, 0) - 1, -1).to(torch.int32)
        inv = torch.empty_like(row)
        inv[order] = row
        source = torch.full((n + 1,), T * k, device="cuda")
        source[torch.where(kept, row.long(), n)] = order  # the last entry takes what has no row
        source = source[:n]
        codes, scale = _quantised(s["x"].float())
        # token T and assignment T * k: the zeros of a row that nothing takes
        codes = torch.cat([codes, codes.new_zeros(1, c["H"])])
        scale = torch.cat([scale, scale.new_zeros(1)])
        token = torch.div(source, k, rounding_mode="floor")
        taken = source < T * k
        return {"recv_x": codes[token], "recv_scale": scale[token], "inv": inv,
                "weight": torch.cat([s["w"].flatten(), scale.new_zeros(1)])[source],
                "src_token": torch.where(taken, token % (T // c["P"]), 0).to(torch.int32),
                "slot": torch.where(taken, source % k, 0).to(torch.int32)}
    p, F = s["plan"], c["F"]
    if s["op"] == "gated":
        gu = _product(p, s["x"].float() * s["xs"][:, None], s["w13"], s["w13s"])
        codes, scale = _quantised(_silu32(gu[:, :F]) * gu[:, F:])
        return {"hid": codes.to(torch.bfloat16), "hid_scale": scale}
    return {"y": _product(p, s["hid"].float() * s["hids"][:, None], s["w2"],
                          s["w2s"]).to(torch.bfloat16)}


# ---- the definition in 64 bits --------------------------------------------
def exact(case, seed):
    """The same outputs from the definition: expert by expert, whole sums of the codes, then
    the scales, in 64 bits. The dispatch's codes and indices are whole numbers (None)."""
    if work(case)["flops"] > 8e12:  # over some 10 s at the card's 64-bit rate
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "dispatch":
        T, k = case["T"], case["k"]
        scale64 = s["x"].double().abs().amax(1) / 127
        scale, weight = [], []
        flat, empty = s["ids"].flatten(), torch.zeros(s["rows"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            at = (flat == e).nonzero().flatten()
            at = at[:case["cap"]] if case["cap"] else at
            scale.append(scale64[at // k])
            weight.append(s["w"].double().flatten()[at])
        return {"recv_x": None, "recv_scale": torch.cat([*scale, empty])[:s["rows"]], "inv": None,
                "weight": torch.cat([*weight, empty])[:s["rows"]], "src_token": None,
                "slot": None}
    E, F, H, R = case["E"], case["F"], case["H"], s["plan"]["rows"]
    a, a_scale, w, w_scale = ((s["x"], s["xs"], s["w13"], s["w13s"]) if case["op"] == "gated" else
                              (s["hid"], s["hids"], s["w2"], s["w2s"]))
    out = torch.zeros(R, w.shape[1], dtype=torch.float64, device="cuda")
    for e, lo, hi in s["plan"]["spans"]:
        whole = a[lo:hi].double() @ w[e].double().T
        out[lo:hi] = whole * a_scale[lo:hi, None].double() * w_scale[e][None, :].double()
    if case["op"] == "down":
        return {"y": out}
    h = out[:, :F] * torch.sigmoid(out[:, :F]) * out[:, F:]
    scale = h.abs().amax(1) / 127
    return {"hid": (h / scale.clamp_min(1e-300)[:, None]).round(), "hid_scale": scale}
