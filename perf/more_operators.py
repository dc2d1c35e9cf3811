"""What a rank does with rows and shards around the collectives of a sharded training step: layer norm with
the residual's addition, and its backward pass; tokens' rows sorted by the experts that a rank holds, and
back with weights, and their gradients; and AdamW over all tensors of a rank's share, with states in 32 or
in 8 bits.  Cases of their real use, their plain forms, and the framework's calls."""
import math
import random

import torch

own = False

EPS = 1e-5                                   # of the norm
E4M3_MAX, SCALE_MIN = 448.0, 2.0 ** -100
BETAS, ADAM_EPS, LR, DECAY, BLOCK = (0.9, 0.95), 1e-8, 1e-4, 0.1, 128
STEP = 1000                                  # steps that the optimizer has behind it
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def listed():
    norm = dict(op="norm", x="bf16", residual="bf16", weight="bf16", y="bf16", group=0, pad=0)
    grad = dict(op="norm_grad", x="bf16", residual="bf16", weight="bf16", pad=0)
    rows = dict(experts=64, of=64, first=0, top_k=8, align=1, x="bf16", group=0)
    return [
        # one request's new token, to 8 bits for the gather
        dict(norm, name="norm_token", rows=1, cols=4096, y="e4m3"),
        # the rows of a 4-rank chunked all-gather's buffer, to 8 bits with a scale per 128 columns
        dict(norm, name="norm_gather", rows=16384, cols=4096, y="e4m3", group=128),
        # odd sizes in f32, nothing 16-byte aligned
        dict(grad, name="norm_grad_odd", rows=1021, cols=5001, x="f32", residual="f32", weight="f32", pad=3),
        # a whole training block
        dict(grad, name="norm_grad_block", rows=16384, cols=4096),
        # a decode batch of odd size on one of eight ranks: its 16 experts of 128, 8-bit rows with their scales
        dict(rows, name="dispatch_batch", op="dispatch", tokens=37, cols=4096, of=128, experts=16, first=32, x="e4m3", group=128),
        # a training block's tokens to all of 64 experts, each one's rows filled up to the products' tiles
        dict(rows, name="dispatch_block", op="dispatch", tokens=16384, cols=4096, align=128),
        # the decode batch's way back, and the block's
        dict(rows, name="combine_batch", op="combine", tokens=37, cols=4096, of=128, experts=16, first=32, weights=True),
        dict(rows, name="combine_block", op="combine", tokens=16384, cols=4096, align=128, weights=True),
        # the gradients of the way back: a rank's quarter of the experts and a width that is no power of two, and the block
        dict(rows, name="combine_grad_share", op="combine_grad", tokens=2000, cols=8064, of=64, experts=16, first=16, top_k=4),
        dict(rows, name="combine_grad_block", op="combine_grad", tokens=16384, cols=4096, align=128),
        # a rank's share of a model's layers: matrices and vectors back to back, 32-bit states and weights, and the
        # weights' bf16 copy for the all-gather
        dict(op="adamw", name="adamw_share", layers=6, width=4096, side=1024, param="f32", grad="bf16", state="f32",
             copy=True, clip=True, stochastic=False),
        # 33 tensors of odd sizes, 8-bit states and bf16 weights, rounded at random
        dict(op="adamw", name="adamw_bytes", count=33, total=32000000, sizes=5, param="bf16", grad="bf16", state="e4m3",
             copy=False, clip=False, stochastic=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "dispatch", "combine", "combine_grad", "adamw", "adamw"))
    if op == "adamw":
        state = rng.choice(("f32", "e4m3"))
        param = rng.choice(("f32", "bf16"))
        return dict(op=op, count=_log(rng, 1, 200), total=_log(rng, 1000, 64000000), sizes=rng.randrange(1 << 20), param=param,
                    grad=rng.choice(("f32", "bf16")), state=state, copy=param == "f32" and rng.random() < 0.5,
                    clip=rng.random() < 0.5, stochastic=state == "e4m3" and rng.random() < 0.7)
    if op in ("norm", "norm_grad"):
        case = dict(op=op, rows=_log(rng, 1, 24000), cols=_log(rng, 64, 8192), x=rng.choice(("bf16", "bf16", "f32")),
                    weight=rng.choice(("bf16", "f32")), pad=rng.choice((0, 0, 1, 8)))
        case["residual"] = "f32" if case["x"] == "f32" else rng.choice(("bf16", "bf16", "f32"))
        if rng.random() < 0.4:               # widths as models have them
            case["cols"] = max(64, case["cols"] // 64 * 64)
        if op == "norm":
            case["y"] = rng.choice(("bf16", "e4m3", "e4m3", "f32" if case["x"] == "f32" else "bf16"))
            case["group"] = rng.choice((0, 32, 64, 128)) if case["y"] == "e4m3" else 0
        return case
    of = _log(rng, 2, 256)
    experts = max(1, of // rng.choice((1, 1, 2, 4, 8)))
    case = dict(op=op, of=of, experts=experts, first=rng.randrange(of - experts + 1), top_k=min(of, rng.choice((1, 2, 3, 4, 6, 8))),
                align=rng.choice((1, 1, 16, 128)), cols=_log(rng, 64, 8192), group=0)
    case["tokens"] = _log(rng, 1, max(1, int(16384 * 8 * 4096 // (case["top_k"] * case["cols"] * (2 if op == "dispatch" else 1)))) // 2)
    case["tokens"] = min(case["tokens"], 40000)
    if rng.random() < 0.5:
        case["cols"] = max(64, case["cols"] // 64 * 64)
    case["x"] = rng.choice(("bf16", "f32", "e4m3") if op == "dispatch" else ("bf16", "bf16", "f32"))
    if case["x"] == "e4m3":
        case["group"] = 128
    if op == "combine":
        case["weights"] = rng.random() < 0.6         # without: the gradient of the dispatch
    return case


# ---- sizes --------------------------------------------------------------------------------------
def _tensors(case):
    """[(elements, whether weights decay)]: matrices do, vectors do not."""
    if "layers" in case:
        w, s = case["width"], case["side"]
        return [(w * w, True), (s * w, True), (s * w, True), (w, False), (w + 1, False)] * case["layers"]
    rng = random.Random(case["sizes"])
    parts = [math.exp(rng.gauss(0.0, 2.0)) for _ in range(case["count"])]
    return [(max(1, int(case["total"] * p / sum(parts))), p > 1.0) for p in parts]


def _starts(case):
    """Where each tensor starts in the flat buffers, and their length: back to back, or in whole blocks of 8-bit states."""
    to, at, starts = (BLOCK if case["state"] == "e4m3" else 1), 0, []
    for n, _ in _tensors(case):
        starts.append(at)
        at += -(-n // to) * to
    return starts, at


def _capacity(case):
    return case["tokens"] * min(case["top_k"], case["experts"]) + case["experts"] * (case["align"] - 1)


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(n for n, _ in _tensors(case))
        p, g = BYTES[case["param"]], BYTES[case["grad"]]
        state = 16 if case["state"] == "f32" else 4 + 16 / BLOCK
        return {"bytes": int(n * (2 * p + g + state + (2 if case["copy"] else 0))), "flops": 16 * n}
    if op in ("norm", "norm_grad"):
        n = case["rows"] * case["cols"]
        x, r, w = (BYTES[case[k]] for k in ("x", "residual", "weight"))
        if op == "norm_grad":                # dy, h, the residual's gradient, dx; weight, both gradients; mean, rstd
            return {"bytes": n * (x + 3 * r) + case["cols"] * (w + 8) + 8 * case["rows"], "flops": 16 * n}
        scales = 0 if case["y"] != "e4m3" else case["rows"] * (-(-case["cols"] // case["group"]) if case["group"] else 1)
        return {"bytes": n * (x + 2 * r + BYTES[case["y"]]) + 2 * case["cols"] * w + 4 * (2 * case["rows"] + scales),
                "flops": 11 * n}
    pairs = case["tokens"] * case["top_k"]
    rows = pairs * case["experts"] / case["of"]          # as many as a rank gets of an even load
    line = case["cols"] * BYTES[case["x"]] + (4 * -(-case["cols"] // case["group"]) if case["group"] else 0)
    few = min(1.0, rows / case["tokens"])                # tokens that the rank's experts take: at most all
    if op == "dispatch":                     # ids in, positions out; each token's row once, each sorted row once
        return {"bytes": int(8 * pairs + (few * case["tokens"] + rows) * line), "flops": 0}
    if op == "combine":
        return {"bytes": int(8 * pairs + (case["tokens"] + rows) * line), "flops": int(2 * rows * case["cols"])}
    return {"bytes": int(12 * pairs + (few * case["tokens"] + 2 * rows) * line), "flops": int(3 * rows * case["cols"])}


# ---- inputs -------------------------------------------------------------------------------------
def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _inputs(case, seed):
    """What the call is given, on the device where there is one: values from the seed alone."""
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]

        def slab(kind, spread, shift=0.0):   # rows of a buffer that is `pad` columns wider
            t = torch.empty(rows, cols + case["pad"], dtype=TYPES[kind], device=dev)
            for i in range(0, rows, 8192):
                t[i:i + 8192] = normal(min(8192, rows - i), cols + case["pad"]) * spread + shift
            return t[:, :cols]

        # a residual stream: a few columns far larger than the rest, and a mean
        outliers = torch.where(torch.rand(cols + case["pad"], generator=g, device=dev) < 0.003, 20.0, 1.0)
        weight = (1.0 + 0.2 * normal(cols)).to(TYPES[case["weight"]])
        if case["op"] == "norm":
            return {"x": slab(case["x"], 0.5), "residual": slab(case["residual"], 2.0 * outliers, 1.5), "weight": weight,
                    "bias": (0.1 * normal(cols)).to(TYPES[case["weight"]])}
        h = slab(case["residual"], 2.0 * outliers, 1.5)
        mean = torch.cat([p.float().mean(-1) for p in h.split(8192)])
        rstd = torch.cat([(p.float().var(-1, unbiased=False) + EPS).rsqrt() for p in h.split(8192)])
        return {"dy": slab(case["x"], 1e-2), "h": h, "dres": slab(case["residual"], 1e-2), "weight": weight,
                "mean": mean, "rstd": rstd}

    if case["op"] == "adamw":
        starts, total = _starts(case)
        p, gr = torch.zeros(total, device=dev), torch.zeros(total, device=dev)
        m, v = torch.zeros(total, device=dev), torch.zeros(total, device=dev)
        for at, (n, _) in zip(starts, _tensors(case)):
            # tensors whose gradients differ by orders of magnitude, and a sixteenth of the elements that have had none
            size = 10.0 ** float(torch.empty(1).uniform_(-5, -2, generator=torch.Generator().manual_seed(seed + at)))
            spread = torch.exp(normal(n))
            spread[torch.rand(n, generator=g, device=dev) < 1 / 16] = 0.0
            p[at:at + n] = 0.02 * normal(n)
            gr[at:at + n] = size * spread * normal(n)
            m[at:at + n] = 0.3 * size * spread * normal(n)
            v[at:at + n] = (size * spread) ** 2 * (0.5 + torch.rand(n, generator=g, device=dev))
        made = {"param": p.to(TYPES[case["param"]]), "grad": gr.to(TYPES[case["grad"]]), "m": m, "v": v}
        if case["state"] == "e4m3":          # as a step before this one has left them: codes, and a scale per 128
            for k, x in (("m", m), ("v", v.sqrt())):
                x = x.view(-1, BLOCK)
                scale = (x.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
                q = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
                if k == "v":
                    q = torch.where(q > 0, q.clamp_min(2.0 ** -9), q)
                made[k], made[k + "_scales"] = q.to(torch.float8_e4m3fn).view(-1), scale
        if case["clip"]:                     # what clipping by the gradients' norm multiplies them with
            made["grad_scale"] = torch.full((1,), 0.37, device=dev)
        return made

    tokens, k, of, cols = case["tokens"], case["top_k"], case["of"], case["cols"]
    # a router's choice: some experts are liked more than others; a few tokens of a padded batch have none
    ids = torch.cat([(normal(n, of) + bias).topk(k, dim=1).indices for bias in [0.7 * normal(of)]
                     for n in [min(8192, tokens - i) for i in range(0, tokens, 8192)]]).to(torch.int32)
    ids[torch.rand(tokens, generator=g, device=dev) < 0.02] = -1
    made = {"ids": ids}

    def slab(rows, spread):
        t = torch.empty(rows, cols, dtype=TYPES[case["x"]], device=dev)
        for i in range(0, rows, 8192):
            t[i:i + 8192] = normal(min(8192, rows - i), cols) * spread
        return t

    if case["op"] == "dispatch":
        made["x"] = slab(tokens, 30.0 if case["x"] == "e4m3" else 1.0)
        if case["group"]:
            made["scales"] = 1e-3 * torch.rand(tokens, -(-cols // case["group"]), generator=g, device=dev)
        return made
    made["position"], made["offsets"], made["counts"] = _route(case, ids)
    made["rows"] = slab(_capacity(case), 1.0)
    if case["op"] == "combine_grad" or case["weights"]:
        made["weights"] = torch.softmax(normal(tokens, k), dim=1)
    if case["op"] == "combine_grad":
        made["dout"] = slab(tokens, 1e-2)
    return made


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    dev = _device()

    def new(kind, *shape):
        return torch.zeros(*shape, dtype=TYPES.get(kind, kind), device=dev)

    # the buffers that a training or serving loop keeps for the results
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        if op == "norm_grad":
            s["dx"], s["dweight"], s["dbias"] = new(case["residual"], rows, cols), new("f32", cols), new("f32", cols)
        else:
            s["residual_out"], s["y"] = new(case["residual"], rows, cols), new(case["y"], rows, cols)
            s["mean"], s["rstd"], s["scales"] = new("f32", rows), new("f32", rows), None
            if case["y"] == "e4m3":
                s["scales"] = new("f32", rows, -(-cols // case["group"]) if case["group"] else 1)
    elif op == "adamw":
        s["step"] = STEP
        if case["copy"]:
            s["copy"] = s["param"].to(torch.bfloat16)
    else:
        tokens, cols = case["tokens"], case["cols"]
        if op == "dispatch":
            s["rows"] = new(case["x"], _capacity(case), cols)
            s["position"] = new(torch.int32, tokens, case["top_k"])
            s["offsets"], s["counts"] = new(torch.int32, case["experts"] + 1), new(torch.int32, case["experts"])
            if case["group"]:
                s["row_scales"] = new("f32", _capacity(case), s["scales"].shape[1])
        elif op == "combine":
            s["out"] = new(case["x"], tokens, cols)
        else:
            s["drows"], s["dweights"] = new(case["x"], _capacity(case), cols), new("f32", tokens, case["top_k"])
    if own:
        import device_triggered_transfers_gb300 as D
        s["stream"] = torch.cuda.current_stream()
        if op in ("norm", "norm_grad"):
            s["op"] = D.LayerNorm(case["cols"], x=case["x"], residual=case["residual"], weight=case["weight"],
                                  y=case.get("y", case["x"]), group=case.get("group", 0), eps=EPS)
        elif op == "adamw":
            starts, _ = _starts(case)
            sizes = _tensors(case)

            def views(t, to=1):
                return None if t is None else [t[at // to:at // to + -(-n // to)] for at, (n, _) in zip(starts, sizes)]

            s["op"] = D.AdamW(views(s["param"]), views(s["grad"]), views(s["m"]), views(s["v"]),
                              m_scales=views(s.get("m_scales"), BLOCK), v_scales=views(s.get("v_scales"), BLOCK),
                              copies=views(s.get("copy")), betas=BETAS, eps=ADAM_EPS,
                              weight_decay=[DECAY if decays else 0.0 for _, decays in sizes],
                              seed=seed if case["stochastic"] else None)
        else:
            s["op"] = D.ExpertRows(case["experts"], case["top_k"], first=case["first"], align=case["align"])
    elif op == "adamw":                      # of each element: its tensor's decay, and its place there for the rounding
        starts, total = _starts(case)
        sizes = torch.tensor([b - a for a, b in zip(starts, starts[1:] + [total])], device=dev)
        s["decay"] = torch.tensor([DECAY if d else 0.0 for _, d in _tensors(case)], device=dev).repeat_interleave(sizes)
        if case["stochastic"]:
            s["numbers"] = torch.arange(len(starts), device=dev)
            s["tensor"] = s["numbers"].repeat_interleave(sizes)
            s["index"] = torch.arange(total, device=dev) - torch.tensor(starts, device=dev).repeat_interleave(sizes)
            s["seed"] = seed
    return s


# ---- the framework's calls ------------------------------------------------------------------------
def _own(s):
    case, op, stream = s["case"], s["op"], s["stream"]
    if case["op"] == "norm":
        op.forward(s["x"], s["weight"], s["bias"], s["y"], residual=s["residual"], residual_out=s["residual_out"],
                   scales=s["scales"], mean=s["mean"], rstd=s["rstd"], stream=stream)
        out = {"y": s["y"], "residual": s["residual_out"], "mean": s["mean"], "rstd": s["rstd"]}
        if case["y"] == "e4m3":
            out["scales"] = s["scales"]
        return out
    if case["op"] == "norm_grad":
        op.backward(s["dy"], s["h"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"], dres=s["dres"],
                    stream=stream)
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if case["op"] == "adamw":
        s["step"] += 1
        op.run(LR, s["step"], grad_scale=s.get("grad_scale"), stream=stream)
        return {k: s[k] for k in ("param", "m", "v", "m_scales", "v_scales", "copy") if k in s}
    if case["op"] == "dispatch":
        op.route(s["ids"], s["position"], s["offsets"], s["counts"], max_rows=s["rows"].shape[0], stream=stream)
        op.dispatch(s["x"], s["position"], s["offsets"], s["counts"], s["rows"], scales=s.get("scales"),
                    row_scales=s.get("row_scales"), stream=stream)
        return {k: s[k] for k in ("position", "offsets", "counts", "rows", "row_scales") if k in s}
    if case["op"] == "combine":
        op.combine(s["rows"], s["position"], s["out"], weights=s.get("weights"), stream=stream)
        return {"out": s["out"]}
    op.combine_backward(s["dout"], s["rows"], s["position"], s["weights"], s["offsets"], s["counts"], s["drows"],
                        s["dweights"], stream=stream)
    return {"drows": s["drows"], "dweights": s["dweights"]}


# ---- plain forms ----------------------------------------------------------------------------------
def _mix(x):
    """32 bits from 32 bits (an int, or an int64 tensor)."""
    x = (x ^ (x >> 16)) * 0x85A308D3 & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * 0xB7E15163 & 0xFFFFFFFF
    return x ^ (x >> 16)


def _bits(t):
    return t.view(torch.int32)


def _to_e4m3(x, noise):
    """To e4m3's values: to the nearest, or (noise: 16 bits) up with the probability of what lies below."""
    if noise is not None:
        size = x.abs()
        low = size < 2.0 ** -6                                  # subnormal: the same spacing as just above 2^-6
        t = torch.where(low, size + 2.0 ** -6, size)
        t = (_bits(t) + (noise.to(torch.int32) << 4) & ~0xFFFFF).view(torch.float32)
        x = torch.where(low, t - 2.0 ** -6, t).clamp_max(E4M3_MAX).copysign(x)
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _adamw(s):
    case, (b1, b2) = s["case"], BETAS
    s["step"] += 1
    t = s["step"]
    g = s["grad"].float()
    if case["clip"]:
        g = g * s["grad_scale"]
    bits = state = None
    if case["stochastic"]:
        seeds = _mix(_mix(_mix(s["seed"]) + t & 0xFFFFFFFF) + s["numbers"] & 0xFFFFFFFF)
        bits = _mix(s["index"] * 0x9E3779B9 + seeds[s["tensor"]] & 0xFFFFFFFF)
    if case["state"] == "e4m3":
        m = (s["m"].float().view(-1, BLOCK) * s["m_scales"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scales"][:, None]).view(-1).square()
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    denom = v.sqrt() * (1 / math.sqrt(1 - b2 ** t)) + ADAM_EPS
    p = s["param"].float()
    p = p * (1 - LR * s["decay"]) - (LR / (1 - b1 ** t)) * (m / denom)
    if case["state"] == "e4m3":
        state = {}
        root = v.sqrt()
        for k, x, noise in (("m", m, None if bits is None else bits >> 16), ("v", root, None if bits is None else bits & 0xFFFF)):
            x = x.view(-1, BLOCK)
            top = x.abs().amax(1)
            scale = (top / E4M3_MAX).clamp_min(SCALE_MIN)
            q = _to_e4m3((x * (1 / scale)[:, None]).view(-1), noise)
            if k == "v":                                        # a root above zero stays above zero
                q = torch.where(root > 0, q.float().clamp_min(2.0 ** -9), 0.0).to(torch.float8_e4m3fn)
            state[k], state[k + "_scales"] = q, scale
    else:
        state = {"m": m, "v": v}
    if case["copy"]:
        state["copy"] = p.to(torch.bfloat16)
    if case["param"] == "bf16":
        if bits is not None:
            p = (_bits(p) + ((bits * 0x2E1B2139 & 0xFFFFFFFF) >> 16).to(torch.int32) & ~0xFFFF).view(torch.float32)
        p = p.to(torch.bfloat16)
    s.update(state, param=p)
    return {"param": p, **state}


def _route(case, ids):
    """Each pair's row: the experts' rows one after another (each one's filled up to a multiple of align), in the
    pairs' order; -1 for the experts of others."""
    n, align = case["experts"], case["align"]
    e = ids.reshape(-1).long() - case["first"]
    e = torch.where((e >= 0) & (e < n) & (ids.reshape(-1) >= 0), e, n)
    counts = torch.zeros(n + 1, dtype=torch.int64, device=ids.device).index_add_(0, e, torch.ones_like(e))
    order = torch.argsort(e, stable=True)
    filled = (counts[:n] + align - 1) // align * align
    offsets = torch.cat([filled.new_zeros(1), filled.cumsum(0)])
    first = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rank = torch.empty_like(e)
    rank[order] = torch.arange(e.numel(), device=ids.device)
    place = rank - first[e] + offsets[e]
    position = torch.where(e < n, place, -1).view(ids.shape)
    return position.to(torch.int32), offsets.to(torch.int32), counts[:n].to(torch.int32)


def _put(rows, position, offsets, counts, values, each):
    """rows with values[pair // each] at the pairs' positions, and zeros where an expert's rows are filled up."""
    size, at = rows.shape[0], position.reshape(-1).long()
    pair = torch.full((size + 1,), -1, dtype=torch.int64, device=rows.device)
    pair = pair.scatter(0, torch.where(at >= 0, at, size), torch.arange(at.numel(), device=rows.device))[:size]
    number = torch.arange(size, device=rows.device)
    e = (torch.searchsorted(offsets.long(), number, right=True) - 1).clamp_max(counts.numel() - 1)
    fill = (number < offsets[-1]) & (number >= offsets[e] + counts[e])
    rest = torch.where(fill[:, None], torch.zeros_like(rows[:1]), rows)
    return torch.where((pair >= 0)[:, None], values[pair.clamp_min(0) // each], rest)


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    op = case["op"]
    if op == "adamw":
        return _adamw(s)
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        n = (s["h"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) * rstd + s["dres"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * n).sum(0), "dbias": dy.sum(0)}
    if op == "norm":
        h = s["x"].float() + s["residual"].float()
        mean = h.mean(-1)
        d = h - mean[:, None]
        rstd = (d.square().mean(-1) + EPS).rsqrt()
        y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
        out = {"residual": h.to(s["residual"].dtype), "mean": mean, "rstd": rstd}
        if case["y"] != "e4m3":
            return {**out, "y": y.to(TYPES[case["y"]])}
        rows, cols = y.shape
        group = case["group"] or cols
        count = -(-cols // group)
        y = torch.nn.functional.pad(y, (0, count * group - cols)).view(rows, count, group)
        scales = (y.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
        q = (y / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {**out, "y": q.view(rows, count * group)[:, :cols].contiguous(), "scales": scales}
    k = case["top_k"]
    if op == "dispatch":
        position, offsets, counts = _route(case, s["ids"])
        plan = position, offsets, counts
        raw = torch.uint8 if case["x"] == "e4m3" else TYPES[case["x"]]
        s["rows"] = _put(s["rows"].view(raw), *plan, s["x"].view(raw), k).view(TYPES[case["x"]])
        out = {"position": position, "offsets": offsets, "counts": counts, "rows": s["rows"]}
        if case["group"]:
            out["row_scales"] = s["row_scales"] = _put(s["row_scales"], *plan, s["scales"], k)
        return out
    at = s["position"].long()
    mine = at >= 0
    picked = torch.where(mine[:, :, None], s["rows"][at.clamp_min(0)].float(), 0.0)
    if op == "combine":
        if case["weights"]:
            picked = picked * s["weights"][:, :, None]
        return {"out": picked.sum(1).to(TYPES[case["x"]])}
    dout = s["dout"].float()
    dweights = (picked * dout[:, None]).sum(-1)
    values = (dout[:, None] * s["weights"][:, :, None]).to(TYPES[case["x"]]).view(-1, case["cols"])
    s["drows"] = _put(s["drows"], s["position"], s["offsets"], s["counts"], values, 1)
    return {"drows": s["drows"], "dweights": dweights}


# ---- in 64 bits -------------------------------------------------------------------------------------
def _exact_norm(case, d):
    if case["op"] == "norm_grad":
        rstd, centred = d["rstd"].unsqueeze(1), d["h"] - d["mean"].unsqueeze(1)
        weighted = d["dy"] * d["weight"]
        inner = torch.einsum("rc,rc->r", weighted, centred).unsqueeze(1) / case["cols"]
        whole = torch.einsum("rc->r", weighted).unsqueeze(1) / case["cols"]
        return {"dx": d["dres"] + rstd * (weighted - whole) - rstd ** 3 * inner * centred,
                "dweight": torch.einsum("rc,rc,ro->c", d["dy"], centred, rstd), "dbias": torch.einsum("rc->c", d["dy"])}
    h = d["x"] + d["residual"]
    variance, mean = torch.var_mean(h, dim=1, correction=0)
    rstd = 1.0 / torch.sqrt(variance + EPS)
    y = torch.einsum("rc,r,c->rc", h - mean.unsqueeze(1), rstd, d["weight"]) + d["bias"]
    if case["y"] != "e4m3":
        return {"residual": h, "mean": mean, "rstd": rstd, "y": y}
    parts = y.split(case["group"] or case["cols"], dim=1)
    scales = torch.stack([(p.abs().max(dim=1).values / E4M3_MAX).clamp(min=SCALE_MIN) for p in parts], dim=1)
    # the codes' values before they are rounded to 8 bits
    y = torch.cat([p / scales[:, i:i + 1] for i, p in enumerate(parts)], dim=1)
    return {"residual": h, "mean": mean, "rstd": rstd, "y": y, "scales": scales}


def _exact_adamw(case, d):
    """Tensor by tensor.  Codes and bf16 weights: the values before they are rounded."""
    out = {k: torch.zeros_like(d[k]) for k in d if k != "grad_scale"}
    del out["grad"]
    starts, _ = _starts(case)
    t = STEP + 1
    for at, (n, decays) in zip(starts, _tensors(case)):
        cut = slice(at, at + n)
        g = d["grad"][cut] * (d["grad_scale"] if case["clip"] else 1.0)
        m, v = d["m"][cut], d["v"][cut]
        blocks = slice(at // BLOCK, -(-(at + n) // BLOCK))
        if case["state"] == "e4m3":
            m = m * d["m_scales"][blocks].repeat_interleave(BLOCK)[:n]
            v = (v * d["v_scales"][blocks].repeat_interleave(BLOCK)[:n]) ** 2
        m = m + (1.0 - BETAS[0]) * (g - m)
        v = v + (1.0 - BETAS[1]) * (g ** 2 - v)
        hat = (m / (1.0 - BETAS[0] ** t)) / (torch.sqrt(v / (1.0 - BETAS[1] ** t)) + ADAM_EPS)
        p = d["param"][cut]
        out["param"][cut] = p - LR * (hat + (DECAY * p if decays else 0.0))
        for k, x in (("m", m), ("v", v.sqrt() if case["state"] == "e4m3" else v)):
            if case["state"] == "e4m3":
                rows = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
                scale = (rows.abs().max(dim=1).values / E4M3_MAX).clamp(min=SCALE_MIN)
                out[k + "_scales"][blocks] = scale
                x = (rows / scale.unsqueeze(1)).reshape(-1)[:n]
            out[k][cut] = x
    if case["copy"]:
        out["copy"] = out["param"].clone()
    return out


def _exact_rows(case, s):
    ids, n, k = s["ids"].long() - case["first"], case["experts"], case["top_k"]
    ids = torch.where(s["ids"] < 0, -1, ids)
    if case["op"] == "dispatch":
        x = s["x"].double()
        out = {"rows": x.new_zeros(_capacity(case), case["cols"])}
        if case["group"]:
            out["row_scales"] = x.new_zeros(_capacity(case), s["scales"].shape[1])
        start = 0
        for e in range(n):
            token, choice = (ids == e).nonzero(as_tuple=True)
            out["rows"][start:start + len(token)] = x[token]
            if case["group"]:
                out["row_scales"][start:start + len(token)] = s["scales"].double()[token]
            start += -(-len(token) // case["align"]) * case["align"]
        # whole numbers are compared with the plain form's alone
        return {"position": None, "offsets": None, "counts": None, **out}
    position = s["position"].long()
    token, choice = (position >= 0).nonzero(as_tuple=True)
    row = position[token, choice]
    weight = s["weights"].double()[token, choice] if "weights" in s else torch.ones(len(token), dtype=torch.float64, device=row.device)
    if case["op"] == "combine":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=row.device)
        for part in torch.arange(len(token), device=row.device).split(16384):
            out.index_add_(0, token[part], s["rows"][row[part]].double() * weight[part].unsqueeze(1))
        return {"out": out}
    drows = torch.zeros(_capacity(case), case["cols"], dtype=torch.float64, device=row.device)
    dweights = torch.zeros(case["tokens"], k, dtype=torch.float64, device=row.device)
    for part in torch.arange(len(token), device=row.device).split(16384):
        dout = s["dout"][token[part]].double()
        drows[row[part]] = dout * weight[part].unsqueeze(1)
        dweights[token[part], choice[part]] = torch.einsum("nc,nc->n", dout, s["rows"][row[part]].double())
    return {"drows": drows, "dweights": dweights}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(case, {k: v.double() for k, v in s.items()})
    if case["op"] == "adamw":
        return _exact_adamw(case, {k: v.double() for k, v in s.items()})
    return _exact_rows(case, s)
