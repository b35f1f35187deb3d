"""Cases of the routing, layer-norm and gradient-clipping operators, and their plain forms.

An expert layer sends every token to k experts: the (token, choice) pairs are
sorted by expert, the tokens' rows are laid out in that order for the products
grouped by expert, and the experts' rows come back to their tokens, weighted.
Around it stand a layer norm with its gradients and, at the end of a training
step, the clipping of all gradients by their common norm.

  kind            computes
  sort            slots[t, j]: the row of token t's j-th choice, rows in expert order
                  (ties in token order; -1 for an id that is no expert's), offsets of
                  the experts' rows, order: the pair t * k + j of each row (-1 past the last)
  dispatch        out[slots[t, j]] = x[t]; in 8 bits the scales of x's rows go with them
  combine         y[t] = sum over j of weights[t, j] * rows[slots[t, j]]
                  (without weights: the gradient of dispatch)
  combine_grad    drows[slots[t, j]] = weights[t, j] * dy[t]
                  dweights[t, j] = dy[t] . rows[slots[t, j]]
  layernorm       h = x + residual; y = (h - mean) / sqrt(var + eps) * weight + bias; y in
                  the input's type, or as e4m3 values with a scale per row and 128 columns
  layernorm_grad  the gradients of y and h with respect to x (and the residual), weight and bias
  clip            norm over all gradients; gradients * min(1, max_norm / (norm + 1e-6))
  grad_norm       the norm alone

Where `own` is false `run` computes the plain form in 32 bits; where it is
true it calls the library.
"""

import math

import torch

own = False

BLOCK = 128          # columns that share one scale
E4M3_MAX = 448.0
TINY = 2.0 ** -126   # smallest scale: a block of zeros keeps a finite one
LN_EPS = 1e-5
CLIP_EPS = 1e-6

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---- the cases ---------------------------------------------------------------


def listed():
    return [
        # A few decoded tokens on their way to the experts: nothing but latency.
        {"name": "sort_step", "kind": "sort", "tokens": 16, "k": 4, "groups": 16, "padded": False,
         "ids": "i64"},
        # A prompt's tokens, the last eighth of the batch padding (no expert's).
        {"name": "sort_prompt", "kind": "sort", "tokens": 16384, "k": 8, "groups": 64,
         "padded": True, "ids": "i64"},
        # A training batch's rows into expert order.
        {"name": "dispatch_prompt", "kind": "dispatch", "tokens": 8192, "k": 4, "groups": 16,
         "cols": 4096, "type": "bf16", "padded": False},
        # The same in 8 bits with the rows' scales, as a norm leaves them: the serving form.
        {"name": "dispatch_fp8", "kind": "dispatch", "tokens": 8192, "k": 4, "groups": 32,
         "cols": 4096, "type": "e4m3", "padded": True},
        # One decoded token's experts added up: nothing but latency.
        {"name": "combine_step", "kind": "combine", "tokens": 1, "k": 8, "groups": 16,
         "cols": 4096, "type": "bf16", "padded": False, "weighted": True},
        # The ragged GEMM workload's sizes, padding among the tokens.
        {"name": "combine_ragged", "kind": "combine", "tokens": 5000, "k": 6, "groups": 16,
         "cols": 3000, "type": "f16", "padded": True, "weighted": True},
        # The backward pass of a training batch through the weighted sum.
        {"name": "combine_grad", "kind": "combine_grad", "tokens": 8192, "k": 4, "groups": 16,
         "cols": 2048, "type": "bf16", "padded": False},
        # One decoded token between two layers.
        {"name": "layernorm_step", "kind": "layernorm", "rows": 1, "cols": 4096, "type": "bf16",
         "residual": True, "fp8": False},
        # A prompt's tokens between two layers.
        {"name": "layernorm_prompt", "kind": "layernorm", "rows": 16384, "cols": 4096,
         "type": "bf16", "residual": True, "fp8": False},
        # The backward pass over a training batch's tokens.
        {"name": "layernorm_grad", "kind": "layernorm_grad", "rows": 8192, "cols": 4096,
         "type": "bf16", "residual": True},
        # The gradients of one small layer.
        {"name": "clip_small", "kind": "clip", "tensors": 9, "total": 300000, "type": "mixed"},
        # The gradients of a model's layers, experts among them.
        {"name": "clip_large", "kind": "clip", "tensors": 48, "total": 256000000, "type": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    """A whole multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


MOST_NORM = 16384 * 4096      # the largest listed norm
MOST_ROWS = 8192 * 4 * 4096   # elements of the largest listed rows in expert order


def draw(rng):
    kind = rng.choice(["sort", "dispatch", "dispatch", "combine", "combine", "combine_grad",
                       "layernorm", "layernorm", "layernorm_grad", "clip", "clip", "grad_norm"])
    if kind in ("clip", "grad_norm"):
        n = _log_int(rng, 1, 60)
        return {"kind": kind, "tensors": n, "total": _log_int(rng, 1000 * n, 100000000),
                "type": rng.choice(["f16", "bf16", "f32", "mixed"])}
    # Row lengths odd, even and round; rows from one token to a batch.
    cols = _log_int(rng, 64, 8192, rng.choice([1, 8, 64, 128]))
    dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
    if kind in ("layernorm", "layernorm_grad"):
        c = {"kind": kind, "rows": min(_log_int(rng, 1, 16384), MOST_NORM // cols), "cols": cols,
             "type": dtype, "residual": rng.random() < 0.7}
        if kind == "layernorm":
            c["fp8"] = rng.random() < 0.4
        return c
    c = {"kind": kind, "k": rng.choice([1, 2, 3, 4, 6, 8]), "padded": rng.random() < 0.4,
         "groups": rng.choice([4, 7, 16, 32, 60, 128, 256])}
    if kind == "sort":
        c["tokens"], c["ids"] = _log_int(rng, 1, 16384), rng.choice(["i32", "i64"])
        return c
    most = MOST_ROWS // (c["k"] * cols) // (2 if dtype == "f32" else 1)
    c["tokens"], c["cols"], c["type"] = min(_log_int(rng, 1, 16384), max(1, most)), cols, dtype
    if kind == "dispatch" and rng.random() < 0.4:
        c["type"] = "e4m3"
    if kind == "combine":
        c["weighted"] = rng.random() < 0.7
    return c


# ---- what a program has in hand -----------------------------------------------


def _normal(g, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return t.mul_(scale).to(dtype)


def _activations(g, rows, cols, dtype):
    """Hidden states: normals about a mean of their own, a few columns much larger."""
    t = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand(cols, generator=g, device="cuda") < 0.01
    t *= torch.where(loud, 12.0, 1.0)
    t += 0.5 * torch.randn((rows, 1), generator=g, device="cuda")
    return t.to(dtype)


def _to_e4m3(t):
    return t.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _by_row_blocks(t):
    """e4m3 values and scales of fp32 rows, one scale per row and 128 columns.
    The scales are stored block by block ([blocks][rows]), as a view rows x blocks."""
    rows, cols = t.shape
    nb = blocks(cols)
    pad = torch.nn.functional.pad(t, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    s = (pad.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    q = _to_e4m3((pad / s[..., None]).view(rows, nb * BLOCK)[:, :cols].contiguous())
    return q, s.t().contiguous().t()


def _padding(case):
    """Tokens at the batch's end that are padding."""
    return case["tokens"] // 8 if case["padded"] else 0


def _choices(g, case):
    """Every token's k experts, all different where there are as many: an uneven
    router's choice; padding has none (-1)."""
    t, k, e = case["tokens"], case["k"], case["groups"]
    liked = 0.7 * torch.randn(e, generator=g, device="cuda")
    noise = torch.rand((t, e), generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    ids = (liked - torch.log(-torch.log(noise))).topk(min(k, e), 1).indices
    ids = ids[:, torch.arange(k, device="cuda") % min(k, e)].contiguous()
    pad = _padding(case)
    if pad:
        ids[t - pad:] = -1
    return ids


def _sizes(case):
    """Elements and types of the gradients: a few large weights, many small ones."""
    n, total = case["tensors"], case["total"]
    share = [0.62 ** (i % 7) * (1.0 + (i * 37 % 11) / 11) for i in range(n)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    names = [("bf16", "f32", "f16")[i % 3] if case["type"] == "mixed" else case["type"]
             for i in range(n)]
    return sizes, names


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    s = {"case": c}
    if c["kind"] in ("clip", "grad_norm"):
        sizes, names = _sizes(c)
        s["grads"] = [_normal(g, (n,), TYPES[t], 0.03 / (1 + i % 5))
                      for i, (n, t) in enumerate(zip(sizes, names))]
        if c["kind"] == "clip":
            s["out"] = [torch.empty_like(t) for t in s["grads"]]
        return s
    if c["kind"] in ("layernorm", "layernorm_grad"):
        dt, rows, cols = TYPES[c["type"]], c["rows"], c["cols"]
        s["x"] = _activations(g, rows, cols, dt)
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
        if c["kind"] == "layernorm":
            s["bias"] = _normal(g, (cols,), dt, 0.1)
            s["residual"] = _activations(g, rows, cols, dt) if c["residual"] else None
        else:
            s["dy"] = _normal(g, (rows, cols), dt)
            s["dh"] = _normal(g, (rows, cols), dt) if c["residual"] else None
        return s
    ids = _choices(g, c)
    if c["kind"] == "sort":
        s["experts"] = ids.to(torch.int32) if c["ids"] == "i32" else ids
        return s
    s["slots"] = _sorted(ids, c["groups"])[0]
    t, k, cols, dt = c["tokens"], c["k"], c["cols"], TYPES[c["type"]]
    if c["kind"] == "dispatch":
        if c["type"] == "e4m3":
            s["x"], s["scales"] = _by_row_blocks(_activations(g, t, cols, torch.float32))
            s["out_scales"] = torch.zeros((blocks(cols), t * k), device="cuda").t()
        else:
            s["x"], s["scales"] = _activations(g, t, cols, dt), None
        # Rows past the experts' last one stay as they are.
        s["out"] = torch.zeros((t * k, cols), dtype=dt, device="cuda")
        return s
    s["rows"] = _normal(g, (t * k, cols), dt)
    s["weights"] = torch.rand((t, k), generator=g, device="cuda") + 0.05
    s["weights"] /= s["weights"].sum(1, keepdim=True)
    if c["kind"] == "combine_grad":
        s["dy"] = _normal(g, (t, cols), dt)
        s["drows"] = torch.zeros_like(s["rows"])
    elif not c["weighted"]:
        s["weights"] = None
    return s


# ---- the plain forms ------------------------------------------------------------


def _sorted(ids, groups):
    """slots, offsets and order of the pairs' experts."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    order = key.argsort(stable=True)
    place = torch.arange(n, device=flat.device)
    slots = torch.empty_like(order)
    slots[order] = place
    slots = torch.where(key < groups, slots, -1)
    counts = torch.zeros(groups + 1, dtype=torch.int64, device=flat.device)
    counts.index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts[:1] * 0, counts[:groups].cumsum(0)])
    order = torch.where(place < offsets[-1], order, -1)
    return slots.view(ids.shape).to(torch.int32), offsets.to(torch.int32), order.to(torch.int32)


def _bytes_of(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_dispatch(s):
    x, slots = _bytes_of(s["x"]), s["slots"].long()
    n, k = slots.numel(), slots.shape[1]
    # Pairs without an expert go to a row of their own, which is dropped.
    place = torch.where(slots < 0, n, slots).reshape(-1)
    out = torch.zeros((n + 1, x.shape[1]), dtype=x.dtype, device=x.device)
    out[place] = x.repeat_interleave(k, 0)
    r = {"rows": out[:n].view(s["x"].dtype)}
    if s["scales"] is not None:
        sc = torch.zeros((n + 1, s["scales"].shape[1]), device=x.device)
        sc[place] = s["scales"].repeat_interleave(k, 0)
        r["scales"] = sc[:n]
    return r


def _plain_combine(s):
    slots = s["slots"].long()
    live = (slots >= 0).float()
    w = live if s["weights"] is None else live * s["weights"]
    r = s["rows"][slots.clamp_min(0)].float()
    return {"y": (r * w[..., None]).sum(1).to(s["rows"].dtype)}


def _plain_combine_grad(s):
    slots, dy = s["slots"].long(), s["dy"].float()
    n = slots.numel()
    r = s["rows"][slots.clamp_min(0)].float()
    dw = (r * dy[:, None, :]).sum(2) * (slots >= 0)
    out = torch.zeros((n + 1, dy.shape[1]), dtype=s["rows"].dtype, device=dy.device)
    out[torch.where(slots < 0, n, slots)] = (s["weights"][..., None] * dy[:, None, :]).to(out.dtype)
    return {"drows": out[:n], "dweights": dw}


def _plain_layernorm(s):
    c = s["case"]
    dt = s["x"].dtype
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["h"] = h.to(dt)
    d = h - h.mean(1, keepdim=True)
    y = d * torch.rsqrt((d * d).mean(1, keepdim=True) + LN_EPS)
    y = y * s["weight"].float() + s["bias"].float()
    if c["fp8"]:
        out["q"], out["scales"] = _by_row_blocks(y)
    else:
        out["y"] = y.to(dt)
    return out


def _plain_layernorm_grad(s):
    h, dy = s["x"].float(), s["dy"].float()
    d = h - h.mean(1, keepdim=True)
    r = torch.rsqrt((d * d).mean(1, keepdim=True) + LN_EPS)
    n = d * r
    g = dy * s["weight"].float()
    dx = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0), "dbias": dy.sum(0)}


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    if s["case"]["kind"] == "grad_norm":
        return {"norm": norm}
    scale = (MAX_NORM / (norm + CLIP_EPS)).clamp_max(1.0)
    return {"norm": norm, "grads": [(g.float() * scale).to(g.dtype) for g in s["grads"]]}


MAX_NORM = 1.0


def run(s):
    c = s["case"]
    kind = c["kind"]
    if not own:
        if kind == "sort":
            slots, offsets, order = _sorted(s["experts"], c["groups"])
            return {"slots": slots, "offsets": offsets, "order": order}
        return {"dispatch": _plain_dispatch, "combine": _plain_combine,
                "combine_grad": _plain_combine_grad, "layernorm": _plain_layernorm,
                "layernorm_grad": _plain_layernorm_grad, "clip": _plain_clip,
                "grad_norm": _plain_clip}[kind](s)
    import tile_size_decision_gb300 as tiles
    if kind == "sort":
        slots, offsets, order = tiles.expert_sort(s["experts"], c["groups"])
        return {"slots": slots, "offsets": offsets, "order": order}
    if kind == "dispatch":
        if s["scales"] is None:
            return {"rows": tiles.expert_dispatch(s["x"], s["slots"], out=s["out"])}
        rows, scales = tiles.expert_dispatch(s["x"], s["slots"], scales=s["scales"], out=s["out"],
                                             scales_out=s["out_scales"])
        return {"rows": rows, "scales": scales}
    if kind == "combine":
        return {"y": tiles.expert_combine(s["rows"], s["slots"], s["weights"])}
    if kind == "combine_grad":
        drows, dw = tiles.expert_combine_grad(s["dy"], s["rows"], s["slots"], s["weights"],
                                              drows_out=s["drows"])
        return {"drows": drows, "dweights": dw}
    if kind == "layernorm":
        if c["fp8"]:
            q, scales, h = tiles.layernorm_fp8(s["x"], s["weight"], s["bias"],
                                               residual=s["residual"], eps=LN_EPS)
            out = {"q": q, "scales": scales}
        else:
            y, h = tiles.layernorm(s["x"], s["weight"], s["bias"], residual=s["residual"],
                                   eps=LN_EPS)
            out = {"y": y}
        if s["residual"] is not None:
            out["h"] = h
        return out
    if kind == "layernorm_grad":
        dx, dw, db = tiles.layernorm_grad(s["dy"], s["x"], s["weight"], eps=LN_EPS, dh=s["dh"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if kind == "grad_norm":
        return {"norm": tiles.grad_norm(s["grads"])}
    norm = tiles.clip_grads(s["grads"], MAX_NORM, eps=CLIP_EPS, out=s["out"])
    return {"norm": norm, "grads": s["out"]}


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    c = case
    if c["kind"] in ("clip", "grad_norm"):
        sizes, names = _sizes(c)
        b = sum(n * BYTES[t] for n, t in zip(sizes, names))
        if c["kind"] == "grad_norm":
            return {"bytes": b + 4, "flops": 2 * sum(sizes)}
        return {"bytes": 2 * b + 4, "flops": 3 * sum(sizes)}
    if c["kind"] == "layernorm":
        e, nb, eb = c["rows"] * c["cols"], c["rows"] * blocks(c["cols"]), BYTES[c["type"]]
        b = e * eb * (3 if c["residual"] else 1) + 2 * c["cols"] * eb
        return {"bytes": b + (e + 4 * nb if c["fp8"] else e * eb), "flops": 8 * e}
    if c["kind"] == "layernorm_grad":
        e, eb = c["rows"] * c["cols"], BYTES[c["type"]]
        return {"bytes": e * eb * (4 if c["residual"] else 3) + c["cols"] * (eb + 8),
                "flops": 16 * e}
    t, k = c["tokens"], c["k"]
    pairs = t * k
    if c["kind"] == "sort":
        return {"bytes": pairs * ((4 if c["ids"] == "i32" else 8) + 8) + 4 * (c["groups"] + 1),
                "flops": pairs}
    live, cols, eb = t - _padding(c), c["cols"], BYTES[c["type"]]
    if c["kind"] == "dispatch":
        row = cols * eb + (4 * blocks(cols) if c["type"] == "e4m3" else 0)
        return {"bytes": 4 * pairs + live * (1 + k) * row, "flops": 0}
    if c["kind"] == "combine":
        b = 4 * pairs + (4 * live * k if c["weighted"] else 0) + (live * k + t) * cols * eb
        return {"bytes": b, "flops": 2 * live * k * cols}
    return {"bytes": 12 * pairs + live * (1 + 2 * k) * cols * eb, "flops": 3 * live * k * cols}


# ---- the definitions in 64 bits ----------------------------------------------------


def _e4m3_grid(v):
    """v rounded to the nearest e4m3 value (ties to even), in 64 bits."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    exponent = torch.frexp(v.abs())[1].double() - 1
    step = torch.exp2(exponent.clamp_min(-6.0) - 3)
    return torch.round(v / step) * step


def _exact_norm(s, case):
    h = s["x"].double()
    out = {}
    if s["residual"] is not None:
        h += s["residual"].double()
        out["h"] = h.clone()
    cols = case["cols"]
    h -= h.sum(1, keepdim=True) / cols
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / cols + LN_EPS)
    y *= s["weight"].double()
    y += s["bias"].double()
    if not case["fp8"]:
        out["y"] = y
        return out
    scales = torch.empty((case["rows"], blocks(cols)), dtype=torch.float64, device=y.device)
    q = torch.empty_like(y)
    for t in range(blocks(cols)):
        part = y[:, t * BLOCK:(t + 1) * BLOCK]
        scales[:, t] = torch.clamp(part.abs().max(1).values / E4M3_MAX, min=TINY)
        q[:, t * BLOCK:(t + 1) * BLOCK] = _e4m3_grid(part / scales[:, t:t + 1])
    out["q"], out["scales"] = q, scales
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind == "sort":
        return None                      # whole numbers
    s = prepare(case, seed)
    if kind in ("clip", "grad_norm"):
        norm = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in s["grads"]:
            norm += torch.dot(g.double(), g.double())
        norm = norm.sqrt()
        if kind == "grad_norm":
            return {"norm": norm}
        scale = min(1.0, MAX_NORM / (float(norm) + CLIP_EPS))
        return {"norm": norm, "grads": [g.double() * scale for g in s["grads"]]}
    if kind == "layernorm":
        return _exact_norm(s, case)
    if kind == "layernorm_grad":
        # y_j = w_j d_j u^(-1/2) + b_j with d = h - mean(h), u = mean(d^2) + eps:
        # du/dh_i = 2 d_i / cols, dd_j/dh_i = [i = j] - 1 / cols.
        cols = case["cols"]
        d, dy, w = s["x"].double(), s["dy"].double(), s["weight"].double()
        d -= d.sum(1, keepdim=True) / cols
        u = d.square().sum(1, keepdim=True) / cols + LN_EPS
        g = dy * w
        dx = (g - g.sum(1, keepdim=True) / cols) / u.sqrt()
        dx -= d * (g * d).sum(1, keepdim=True) / (cols * u * u.sqrt())
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dweight": (dy * d / u.sqrt()).sum(0), "dbias": dy.sum(0)}
    slots = s["slots"]
    if kind == "dispatch":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        nb = blocks(case["cols"])
        scales = torch.zeros((slots.numel(), nb), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = (slots[:, j] >= 0).nonzero()[:, 0]
            out[slots[t, j].long()] = s["x"].double()[t]
            if s["scales"] is not None:
                scales[slots[t, j].long()] = s["scales"].double()[t]
        return {"rows": out} if s["scales"] is None else {"rows": out, "scales": scales}
    if kind == "combine":
        y = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = (slots[:, j] >= 0).nonzero()[:, 0]
            part = s["rows"][slots[t, j].long()].double()
            if s["weights"] is not None:
                part *= s["weights"][t, j].double()[:, None]
            y[t] += part
        return {"y": y}
    drows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros((case["tokens"], case["k"]), dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        t = (slots[:, j] >= 0).nonzero()[:, 0]
        at, dy = slots[t, j].long(), s["dy"][t].double()
        drows[at] = dy * s["weights"][t, j].double()[:, None]
        dw[t, j] = (dy * s["rows"][at].double()).sum(1)
    return {"drows": drows, "dweights": dw}
