"""The operators that a rank runs on the block it owns, between a reduce-scatter and an all-gather:
the residual's addition with a root-mean-square norm (output in bf16, f32 or 8 bits with scales),
that norm's backward pass, and the orthogonalisation of a momentum update by Newton-Schulz
products.  Cases of their real use, their plain forms, and the framework's calls."""
import math

import torch

own = False

EPS = 1e-6                                   # of the norm
ORTHO_EPS = 1e-7                             # added to the update's Frobenius norm
STEPS, COEFFS = 5, (3.4445, -4.7750, 2.0315)   # Newton-Schulz quintic
MU = 0.95                                    # momentum
E4M3_MAX, SCALE_MIN = 448.0, 2.0 ** -100
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def listed():
    norm = dict(op="norm", x="bf16", residual="bf16", weight="bf16", y="bf16", group=0, pad=0)
    grad = dict(op="norm_grad", x="bf16", residual="bf16", weight="bf16", pad=0)
    ortho = dict(op="ortho", x="bf16", batch=1, momentum=False)
    return [
        # one request's new token, the rows' 8 bits scaled row by row
        dict(norm, name="norm_token", rows=1, cols=4096, y="e4m3"),
        # a decode batch of odd size at a width that is no power of two, scales per 128 columns
        dict(norm, name="norm_batch", rows=37, cols=8064, y="e4m3", group=128),
        # a prompt's rows, bf16 out
        dict(norm, name="norm_prompt", rows=2048, cols=4096),
        # odd sizes, f32 residual stream, x a slice of a wider buffer: nothing is 16-byte aligned
        dict(norm, name="norm_odd", rows=4093, cols=5001, residual="f32", pad=7),
        # the rows of a 4-rank chunked all-gather's buffer, to 8 bits for the gather
        dict(norm, name="norm_gather", rows=16384, cols=4096, y="e4m3", group=128),
        # the rows of the 8-rank tiled all-gather's buffer
        dict(norm, name="norm_wide", rows=64000, cols=8064, y="e4m3"),
        # the backward pass: a small micro-batch, a whole training block, odd sizes in f32
        dict(grad, name="grad_small", rows=16, cols=4096),
        dict(grad, name="grad_block", rows=16384, cols=4096),
        dict(grad, name="grad_odd", rows=1021, cols=5001, x="f32", residual="f32", weight="f32", pad=3),
        # an odd tall matrix (a small projection's update)
        dict(ortho, name="ortho_small", rows=1000, cols=256),
        # two wide matrices of one rank's share, f32 gradients through a Nesterov momentum
        dict(ortho, name="ortho_momentum", rows=1024, cols=4096, batch=2, x="f32", momentum=True),
        # a large square matrix
        dict(ortho, name="ortho_large", rows=4096, cols=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_grad", "ortho", "ortho"))
    if op == "ortho":
        rows, cols = _log(rng, 48, 4096), _log(rng, 48, 4096)
        big = max(1, int(4e7 // (rows * cols)))
        return dict(op=op, rows=rows, cols=cols, batch=_log(rng, 1, min(8, big)), x=rng.choice(("bf16", "f32")),
                    momentum=rng.random() < 0.5)
    case = dict(op=op, cols=_log(rng, 64, 8192), x=rng.choice(("bf16", "bf16", "f32")),
                weight=rng.choice(("bf16", "f32")), pad=rng.choice((0, 0, 1, 8)))
    case["rows"] = _log(rng, 1, 32768)
    case["residual"] = "f32" if case["x"] == "f32" else rng.choice(("bf16", "bf16", "f32"))
    if rng.random() < 0.4:                   # widths as models have them
        case["cols"] = max(64, case["cols"] // 64 * 64)
    if op == "norm":
        case["y"] = rng.choice(("bf16", "e4m3", "e4m3", "f32" if case["x"] == "f32" else "bf16"))
        case["group"] = rng.choice((0, 32, 64, 128)) if case["y"] == "e4m3" else 0
    return case


def _sides(case):
    return min(case["rows"], case["cols"]), max(case["rows"], case["cols"])


def work(case):
    n = case["rows"] * case["cols"]
    if case["op"] == "ortho":
        s, l = _sides(case)
        b = case["batch"]
        moved = n * (BYTES[case["x"]] + 2 + (8 if case["momentum"] else 0))
        # X X^T and A A are symmetric: half of each is enough; (b A + c A A) X is whole
        return {"bytes": b * moved, "flops": b * STEPS * (s * (s + 1) * l + s * (s + 1) * s + 2 * s * s * l)}
    x, r, w = (BYTES[case[k]] for k in ("x", "residual", "weight"))
    if case["op"] == "norm_grad":            # dy, h, the residual's gradient, dx; weight, rstd, its gradient
        return {"bytes": n * (x + 3 * r) + case["cols"] * (w + 4) + 4 * case["rows"], "flops": 12 * n}
    scales = 0 if case["y"] != "e4m3" else case["rows"] * (-(-case["cols"] // case["group"]) if case["group"] else 1)
    return {"bytes": n * (x + 2 * r + BYTES[case["y"]]) + case["cols"] * w + 4 * (case["rows"] + scales),
            "flops": 8 * n}


def _inputs(case, seed):
    """What the call is given, on the device where there is one: values from the seed alone."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(seed)
    rows, cols = case["rows"], case["cols"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "ortho":
        # a gradient: a few strong directions of falling size over small noise in every direction
        b, k = case["batch"], max(1, min(rows, cols) // 8)
        fall = 1.0 / torch.arange(1, k + 1, device=dev).float().sqrt()
        grad = (normal(b, rows, k) * fall) @ normal(b, k, cols) + 0.3 * normal(b, rows, cols)
        made = {"x": (1e-3 * grad).to(TYPES[case["x"]])}
        if case["momentum"]:
            made["momentum"] = 3e-3 * normal(b, rows, cols)
        return made

    def slab(kind, spread):                  # rows of a buffer that is `pad` columns wider
        t = torch.empty(rows, cols + case["pad"], dtype=TYPES[kind], device=dev)
        for i in range(0, rows, 8192):
            t[i:i + 8192] = normal(min(8192, rows - i), cols + case["pad"]) * spread
        return t[:, :cols]

    # a residual stream has a few columns far larger than the rest
    outliers = torch.where(torch.rand(cols + case["pad"], generator=g, device=dev) < 0.003, 20.0, 1.0)
    weight = (1.0 + 0.2 * normal(cols)).to(TYPES[case["weight"]])
    if case["op"] == "norm":
        return {"x": slab(case["x"], 0.5), "residual": slab(case["residual"], 2.0 * outliers), "weight": weight}
    h = slab(case["residual"], 2.0 * outliers)
    rstd = torch.cat([(p.float().square().mean(-1) + EPS).rsqrt() for p in h.split(8192)])
    return {"dy": slab(case["x"], 1e-2), "h": h, "dres": slab(case["residual"], 1e-2), "weight": weight,
            "rstd": rstd}


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    dev, rows, cols = s["weight" if "weight" in s else "x"].device, case["rows"], case["cols"]

    def new(kind, *shape):
        return torch.empty(*shape, dtype=TYPES[kind], device=dev)

    # the buffers that a training or serving loop keeps for the results
    if case["op"] == "ortho":
        s["out"] = new("bf16", case["batch"], rows, cols)
    elif case["op"] == "norm_grad":
        s["dx"], s["dweight"] = new(case["residual"], rows, cols), new("f32", cols)
    else:
        s["residual_out"], s["y"] = new(case["residual"], rows, cols), new(case["y"], rows, cols)
        s["rstd"] = new("f32", rows)
        s["scales"] = None
        if case["y"] == "e4m3":
            s["scales"] = new("f32", rows, -(-cols // case["group"]) if case["group"] else 1)
    if own:
        import device_triggered_transfers_gb300 as D
        if case["op"] == "ortho":
            s["op"] = D.Orthogonalizer(rows, cols, batch=case["batch"], dtype=case["x"], steps=STEPS, coeffs=COEFFS,
                                       eps=ORTHO_EPS, mu=MU if case["momentum"] else None, nesterov=True)
        else:
            s["op"] = D.RMSNorm(cols, x=case["x"], residual=case["residual"], weight=case["weight"],
                                y=case.get("y", case["x"]), group=case.get("group", 0), eps=EPS)
        s["stream"] = torch.cuda.current_stream()
    return s


def _own(s):
    case, op = s["case"], s["op"]
    if case["op"] == "ortho":
        if case["momentum"]:
            op.run(s["x"], s["out"], momentum=s["momentum"], stream=s["stream"])
            return {"out": s["out"], "momentum": s["momentum"]}
        op.run(s["x"], s["out"], stream=s["stream"])
        return {"out": s["out"]}
    if case["op"] == "norm_grad":
        op.backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], dres=s["dres"], stream=s["stream"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    op.forward(s["x"], s["weight"], s["y"], residual=s["residual"], residual_out=s["residual_out"],
               scales=s["scales"], rstd=s["rstd"], stream=s["stream"])
    out = {"y": s["y"], "residual": s["residual_out"], "rstd": s["rstd"]}
    if case["y"] == "e4m3":
        out["scales"] = s["scales"]
    return out


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    if case["op"] == "ortho":
        out = {}
        u = s["x"].float()
        if case["momentum"]:
            s["momentum"].mul_(MU).add_(u)
            u = u + MU * s["momentum"]
            out["momentum"] = s["momentum"]
        tall = case["rows"] > case["cols"]
        x = u.transpose(1, 2) if tall else u
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + ORTHO_EPS)
        a, b, c = COEFFS
        for _ in range(STEPS):
            gram = x @ x.transpose(1, 2)
            x = a * x + (b * gram + c * (gram @ gram)) @ x
        out["out"] = (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()
        return out
    w = s["weight"].float()
    if case["op"] == "norm_grad":
        dy = s["dy"].float()
        xh = s["h"].float() * s["rstd"][:, None]
        wdy = dy * w
        dx = (wdy - xh * (wdy * xh).mean(-1, keepdim=True)) * s["rstd"][:, None] + s["dres"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * xh).sum(0)}
    h = s["x"].float() + s["residual"].float()
    rstd = (h.square().mean(-1) + EPS).rsqrt()
    y = h * rstd[:, None] * w
    out = {"residual": h.to(s["residual"].dtype), "rstd": rstd}
    if case["y"] != "e4m3":
        return {**out, "y": y.to(TYPES[case["y"]])}
    rows, cols = y.shape
    group = case["group"] or cols
    count = -(-cols // group)
    y = torch.nn.functional.pad(y, (0, count * group - cols)).view(rows, count, group)
    scales = (y.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (y / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {**out, "y": q.view(rows, count * group)[:, :cols].contiguous(), "scales": scales}


def exact(case, seed):
    s = _inputs(case, seed)
    d = {k: v.double() for k, v in s.items()}
    if case["op"] == "ortho":
        out, u = {}, d["x"]
        if case["momentum"]:
            out["momentum"] = d["momentum"] * MU + u
            u = u + out["momentum"] * MU
        results = []
        for m in u:
            m = m if m.shape[0] <= m.shape[1] else m.T
            m = m / (torch.linalg.matrix_norm(m) + ORTHO_EPS)
            eye = torch.eye(m.shape[0], dtype=torch.float64, device=m.device)
            for _ in range(STEPS):
                gram = m @ m.T
                m = torch.addmm(COEFFS[0] * eye, COEFFS[1] * eye + COEFFS[2] * gram, gram) @ m
            results.append(m if case["rows"] <= case["cols"] else m.T)
        return {**out, "out": torch.stack(results)}
    if case["op"] == "norm_grad":
        rstd = d["rstd"].unsqueeze(1)
        weighted = d["dy"] * d["weight"]
        inner = torch.einsum("rc,rc->r", weighted, d["h"]).unsqueeze(1) / case["cols"]
        dweight = torch.einsum("rc,rc->c", d["dy"], d["h"] * rstd)
        return {"dx": d["dres"] + rstd * weighted - rstd ** 3 * inner * d["h"], "dweight": dweight}
    h = d["x"] + d["residual"]
    rstd = 1.0 / torch.sqrt(torch.einsum("rc,rc->r", h, h) / case["cols"] + EPS)
    y = torch.einsum("rc,r,c->rc", h, rstd, d["weight"])
    if case["y"] != "e4m3":
        return {"residual": h, "rstd": rstd, "y": y}
    parts = y.split(case["group"] or case["cols"], dim=1)
    scales = torch.stack([(p.abs().max(dim=1).values / E4M3_MAX).clamp(min=SCALE_MIN) for p in parts], dim=1)
    # the codes' values before they are rounded to 8 bits
    y = torch.cat([p / scales[:, i:i + 1] for i, p in enumerate(parts)], dim=1)
    return {"residual": h, "rstd": rstd, "y": y, "scales": scales}
