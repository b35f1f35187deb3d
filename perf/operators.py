"""Cases of the 8-bit and expert-layer operators, and their plain forms.

A transformer block that serves or trains with this library's products runs
them in this order: the residual sum and its root-mean-square norm, whose
output leaves in 8 bits with one scale per row and 128 columns; a dense
product of such rows with an 8-bit weight that has one scale per 128 x 128
block; and products grouped by expert, where every expert multiplies its own
run of rows by its own weight, in 16 bits (with both gradients) or in 8 bits.

  kind      computes
  norm      h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; y in the
            input's type, or as e4m3 values with a scale per row and block of 128
  norm_grad the gradients of y and h with respect to x (and the residual) and weight
  fp8       c[m, n] = sum over blocks t of 128 of
            sa[m, t] * sb[n / 128, t] * sum_k in t a[m, k] * b[n, k]
  grouped   c[i] = a[i] @ w[e] for the rows i of expert e        (w: E x K x N)
  dgrad     da[i] = dc[i] @ w[e]^T
  wgrad     dw[e] = sum over the rows i of expert e of a[i]^T dc[i]
  fp8_grouped  the 8-bit product with a weight and block scales per expert

Where `own` is false `run` computes the plain form in 32 bits; where it is
true it calls the library.
"""

import math

import torch

own = False

BLOCK = 128          # columns (and weight rows) that share one scale
E4M3_MAX = 448.0
TINY = 2.0 ** -126   # smallest scale: a block of zeros keeps a finite one
EPS = 1e-6

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---- the cases ---------------------------------------------------------------


def listed():
    return [
        # One decoded token between two layers: nothing but latency.
        {"name": "norm_step", "kind": "norm", "rows": 1, "cols": 4096, "type": "bf16",
         "residual": True, "fp8": True},
        # A prompt's tokens between two layers, on the way into an 8-bit product.
        {"name": "norm_prompt", "kind": "norm", "rows": 16384, "cols": 4096, "type": "bf16",
         "residual": True, "fp8": True},
        # The sizes of the ragged GEMM workload: rows whose length is no power of two, 16 bits out.
        {"name": "norm_ragged", "kind": "norm", "rows": 5000, "cols": 3000, "type": "f16",
         "residual": False, "fp8": False},
        # The backward pass over a training batch's tokens.
        {"name": "norm_grad", "kind": "norm_grad", "rows": 8192, "cols": 4096, "type": "bf16",
         "residual": True},
        # A few decoded tokens through one dense layer: the weight is read once.
        {"name": "fp8_step", "kind": "fp8", "m": 16, "n": 4096, "k": 4096, "out": "bf16"},
        # The ragged GEMM workload's sizes: the last tile and the last scale block are short.
        {"name": "fp8_ragged", "kind": "fp8", "m": 5000, "n": 3000, "k": 4096, "out": "f32"},
        # The headline GEMM's sizes in 8 bits: a prompt through one dense layer.
        {"name": "fp8_square", "kind": "fp8", "m": 4096, "n": 4096, "k": 4096, "out": "f16"},
        # A few decoded tokens per expert: every expert's weight is read for them.
        {"name": "grouped_step", "kind": "grouped", "tokens": 64, "experts": 16, "k": 2048,
         "n": 2048, "type": "bf16"},
        # The batched GEMM workload's sizes with ragged items, one of them empty: forward ...
        {"name": "grouped_forward", "kind": "grouped", "tokens": 32768, "experts": 16, "k": 1024,
         "n": 2048, "type": "bf16"},
        # ... the gradient of its rows ...
        {"name": "grouped_dgrad", "kind": "dgrad", "tokens": 32768, "experts": 16, "k": 1024,
         "n": 2048, "type": "bf16"},
        # ... and of its weights.
        {"name": "grouped_wgrad", "kind": "wgrad", "tokens": 32768, "experts": 16, "k": 1024,
         "n": 2048, "type": "bf16"},
        # A prompt through the experts in 8 bits.
        {"name": "grouped_fp8", "kind": "fp8_grouped", "tokens": 8192, "experts": 32, "k": 4096,
         "n": 2048, "out": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    """A whole multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


MOST_MNK = 4096 ** 3          # the largest listed product
MOST_NORM = 16384 * 4096      # the largest listed norm


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_grad", "fp8", "fp8", "grouped", "grouped", "dgrad",
                       "wgrad", "fp8_grouped"])
    if kind in ("norm", "norm_grad"):
        # Rows from one token to a batch; row lengths odd, even and round.
        cols = _log_int(rng, 64, 8192, rng.choice([1, 8, 64, 128]))
        rows = min(_log_int(rng, 1, 16384), MOST_NORM // cols)
        c = {"kind": kind, "rows": rows, "cols": cols,
             "type": rng.choice(["f16", "bf16", "bf16", "f32"]), "residual": rng.random() < 0.7}
        if kind == "norm":
            c["fp8"] = rng.random() < 0.6
        return c
    # Contracted lengths are whole 16-byte rows; the 8-bit ones need not end on a block of 128.
    k = _log_int(rng, 128, 4096, rng.choice([16, 64, 128]))
    n = _log_int(rng, 128, 4096, rng.choice([8, 64, 128]))
    if kind == "fp8":
        m = min(_log_int(rng, 1, 8192), MOST_MNK // (k * n))
        return {"kind": kind, "m": m, "n": n, "k": k, "out": rng.choice(["f16", "bf16", "f32"])}
    experts = rng.choice([2, 4, 7, 8, 16, 32])
    tokens = min(_log_int(rng, 1, 32768), MOST_MNK // (k * n))
    c = {"kind": kind, "tokens": tokens, "experts": experts, "k": k, "n": n}
    if kind == "fp8_grouped":
        c["out"] = rng.choice(["f16", "bf16"])
    else:
        c["type"] = rng.choice(["f16", "bf16"])
    return c


# ---- what a program has in hand -----------------------------------------------


def _normal(g, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return t.mul_(scale).to(dtype)


def _activations(g, rows, cols, dtype):
    """Hidden states: unit normals with a few columns an order of magnitude larger."""
    t = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand(cols, generator=g, device="cuda") < 0.01
    t *= torch.where(loud, 12.0, 1.0)
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


def _by_square_blocks(t):
    """e4m3 values and scales of fp32 weights (..., N, K), one scale per 128 x 128."""
    *lead, n, k = t.shape
    nb, kb = blocks(n), blocks(k)
    pad = torch.nn.functional.pad(t, (0, kb * BLOCK - k, 0, nb * BLOCK - n))
    v = pad.view(*lead, nb, BLOCK, kb, BLOCK)
    s = (v.abs().amax((-3, -1)) / E4M3_MAX).clamp_min(TINY)
    q = (v / s[..., :, None, :, None]).view(*lead, nb * BLOCK, kb * BLOCK)[..., :n, :k]
    return _to_e4m3(q.contiguous()), s.contiguous()


def _group_sizes(seed, tokens, experts):
    """Rows of each expert: a router's uneven choice, with one expert left out."""
    g = torch.Generator().manual_seed(seed)
    p = torch.softmax(torch.randn(experts, generator=g) * 0.5, 0)
    out = int(torch.randint(experts, (1,), generator=g))
    if experts > 2:
        p[out] = 0.0
    who = torch.multinomial(p, tokens, replacement=True, generator=g)
    return torch.bincount(who, minlength=experts)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    s = {"case": c}
    if c["kind"] in ("norm", "norm_grad"):
        dt = TYPES[c["type"]]
        rows, cols = c["rows"], c["cols"]
        s["x"] = _activations(g, rows, cols, dt)
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
        if c["kind"] == "norm":
            s["residual"] = _activations(g, rows, cols, dt) if c["residual"] else None
        else:
            s["dy"] = _normal(g, (rows, cols), dt)
            s["dh"] = _normal(g, (rows, cols), dt) if c["residual"] else None
    elif c["kind"] == "fp8":
        m, n, k = c["m"], c["n"], c["k"]
        s["a"], s["sa"] = _by_row_blocks(_activations(g, m, k, torch.float32))
        s["b"], s["sb"] = _by_square_blocks(_normal(g, (n, k), torch.float32, k ** -0.5))
    else:
        t, e, k, n = c["tokens"], c["experts"], c["k"], c["n"]
        sizes = _group_sizes(seed, t, e)
        s["largest"] = max(1, int(sizes.max()))
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(
            torch.int32).cuda()
        if c["kind"] == "fp8_grouped":
            s["a"], s["sa"] = _by_row_blocks(_activations(g, t, k, torch.float32))
            s["b"], s["sb"] = _by_square_blocks(_normal(g, (e, n, k), torch.float32, k ** -0.5))
        else:
            dt = TYPES[c["type"]]
            if c["kind"] != "dgrad":
                s["a"] = _activations(g, t, k, dt)
            if c["kind"] != "grouped":
                s["dc"] = _normal(g, (t, n), dt)
            if c["kind"] != "wgrad":
                s["w"] = _normal(g, (e, k, n), dt, k ** -0.5)
    if own:
        import tile_size_decision_gb300 as tiles
        if c["kind"] == "norm_grad":
            s["workspace"] = tiles.rmsnorm_grad_workspace(s["x"])
        elif c["kind"] != "norm":
            s["workspace"] = tiles.workspace()
    return s


# ---- the plain forms ------------------------------------------------------------


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    dt = TYPES[c["type"]]
    out = {}
    if s["residual"] is not None:
        out["h"] = h.to(dt)
    if c["fp8"]:
        out["q"], out["scales"] = _by_row_blocks(y)
    else:
        out["y"] = y.to(dt)
    return out


def _plain_norm_grad(s):
    h, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    g = dy * w
    dx = r * g - h * (r * r * r) * (g * h).mean(1, keepdim=True)
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h * r).sum(0)}


def _spread(scales, length, dim):
    """A scale per block as a scale per element along dim."""
    return scales.repeat_interleave(BLOCK, dim).narrow(dim, 0, length)


def _plain_fp8(s):
    m, n, k = (s["case"][x] for x in ("m", "n", "k"))
    a = s["a"].float() * _spread(s["sa"], k, 1)
    b = s["b"].float() * _spread(_spread(s["sb"], n, 0), k, 1)
    return {"c": (a @ b.t()).to(TYPES[s["case"]["out"]])}


def _place(s):
    """Each row's expert, and its position among that expert's rows."""
    off = s["offsets"].long()
    row = torch.arange(s["case"]["tokens"], device=off.device)
    e = torch.searchsorted(off, row, right=True) - 1
    return e, row - off[e]


def _padded(s, rows, e, pos):
    """Every expert's rows padded with zeros to the longest run."""
    p = torch.zeros((s["case"]["experts"], s["largest"], rows.shape[1]), device=rows.device)
    p[e, pos] = rows
    return p


def _plain_grouped(s):
    c = s["case"]
    e, pos = _place(s)
    if c["kind"] == "wgrad":
        pa, pd = _padded(s, s["a"].float(), e, pos), _padded(s, s["dc"].float(), e, pos)
        return {"dw": torch.bmm(pa.transpose(1, 2), pd).to(s["a"].dtype)}
    if c["kind"] == "fp8_grouped":
        a = s["a"].float() * _spread(s["sa"], c["k"], 1)
        b = s["b"].float() * _spread(_spread(s["sb"], c["n"], 1), c["k"], 2)
        y = torch.bmm(_padded(s, a, e, pos), b.transpose(1, 2))
        return {"c": y[e, pos].to(TYPES[c["out"]])}
    w = s["w"].float()
    if c["kind"] == "dgrad":
        return {"da": torch.bmm(_padded(s, s["dc"].float(), e, pos),
                                w.transpose(1, 2))[e, pos].to(s["dc"].dtype)}
    return {"c": torch.bmm(_padded(s, s["a"].float(), e, pos), w)[e, pos].to(s["a"].dtype)}


def run(s):
    c = s["case"]
    kind = c["kind"]
    if not own:
        if kind == "norm":
            return _plain_norm(s)
        if kind == "norm_grad":
            return _plain_norm_grad(s)
        return _plain_fp8(s) if kind == "fp8" else _plain_grouped(s)
    import tile_size_decision_gb300 as tiles
    if kind == "norm":
        if c["fp8"]:
            q, scales, h = tiles.rmsnorm_fp8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            out = {"q": q, "scales": scales}
        else:
            y, h = tiles.rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            out = {"y": y}
        if s["residual"] is not None:
            out["h"] = h
        return out
    ws = s["workspace"]
    if kind == "norm_grad":
        dx, dw = tiles.rmsnorm_grad(s["dy"], s["x"], s["weight"], eps=EPS, dh=s["dh"], workspace=ws)
        return {"dx": dx, "dweight": dw}
    if kind == "fp8":
        return {"c": tiles.gemm_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=c["out"],
                                    workspace=ws)}
    if kind == "fp8_grouped":
        return {"c": tiles.grouped_gemm_fp8(s["a"], s["sa"], s["b"], s["sb"], s["offsets"],
                                            out_dtype=c["out"], workspace=ws)}
    if kind == "grouped":
        return {"c": tiles.grouped_gemm(s["a"], s["w"], s["offsets"], workspace=ws)}
    if kind == "dgrad":
        return {"da": tiles.grouped_gemm(s["dc"], s["w"], s["offsets"], trans_b=True,
                                         workspace=ws)}
    return {"dw": tiles.grouped_wgrad(s["a"], s["dc"], s["offsets"], workspace=ws)}


# ---- what a pass cannot do without ------------------------------------------------


def work(case):
    c = case
    if c["kind"] == "norm":
        e, nb, eb = c["rows"] * c["cols"], c["rows"] * blocks(c["cols"]), BYTES[c["type"]]
        b = e * eb * (3 if c["residual"] else 1) + c["cols"] * eb
        b += e + 4 * nb if c["fp8"] else e * eb
        return {"bytes": b, "flops": 6 * e}
    if c["kind"] == "norm_grad":
        e, eb = c["rows"] * c["cols"], BYTES[c["type"]]
        return {"bytes": e * eb * (4 if c["residual"] else 3) + c["cols"] * (eb + 4),
                "flops": 12 * e}
    if c["kind"] == "fp8":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * k + 4 * (m + blocks(n)) * blocks(k) + m * n * BYTES[c["out"]],
                "flops": 2 * m * n * k}
    t, e, k, n = c["tokens"], c["experts"], c["k"], c["n"]
    # Experts that have rows: one of more than two is left out.
    full = min(t, e - 1 if e > 2 else e)
    if c["kind"] == "fp8_grouped":
        b = t * k + 4 * t * blocks(k) + full * (n * k + 4 * blocks(n) * blocks(k))
        b += t * n * BYTES[c["out"]]
    elif c["kind"] == "wgrad":
        b = t * (k + n) * 2 + e * k * n * 2
    else:
        b = t * (k + n) * 2 + full * k * n * 2
    return {"bytes": b + 4 * (e + 1), "flops": 2 * t * k * n}


# ---- the definitions in 64 bits ----------------------------------------------------


def _e4m3_grid(v):
    """v rounded to the nearest e4m3 value (ties to even), in 64 bits."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    exponent = torch.frexp(v.abs())[1].double() - 1
    step = torch.exp2(exponent.clamp_min(-6.0) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            h += s["residual"].double()
            out["h"] = h
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["cols"] + EPS)
        y *= s["weight"].double()
        if not case["fp8"]:
            out["y"] = y
            return out
        scales = torch.empty((case["rows"], blocks(case["cols"])), dtype=torch.float64,
                             device=y.device)
        q = torch.empty_like(y)
        for t in range(blocks(case["cols"])):
            part = y[:, t * BLOCK:(t + 1) * BLOCK]
            scales[:, t] = torch.clamp(part.abs().max(1).values / E4M3_MAX, min=TINY)
            q[:, t * BLOCK:(t + 1) * BLOCK] = _e4m3_grid(part / scales[:, t:t + 1])
        out["q"], out["scales"] = q, scales
        return out
    if kind == "norm_grad":
        # y_j = w_j h_j u^(-1/2), u = mean(h^2) + eps: dy_j / dh_i has the term
        # -w_j h_j h_i u^(-3/2) / cols.
        h, dy, w = s["x"].double(), s["dy"].double(), s["weight"].double()
        u = h.square().sum(1, keepdim=True) / case["cols"] + EPS
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = dy * w / u.sqrt() - h * dot / (case["cols"] * u * u.sqrt())
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dweight": (dy * h / u.sqrt()).sum(0)}
    if kind in ("fp8", "fp8_grouped"):
        off = s["offsets"].tolist() if kind == "fp8_grouped" else [0, case["m"]]
        rows = off[-1]
        c = torch.zeros((rows, case["n"]), dtype=torch.float64, device="cuda")
        nrow = torch.arange(case["n"], device="cuda") // BLOCK
        for e in range(len(off) - 1):
            lo, hi = off[e], off[e + 1]
            b, sb = (s["b"][e], s["sb"][e]) if kind == "fp8_grouped" else (s["b"], s["sb"])
            for t in range(blocks(case["k"]) if hi > lo else 0):
                kk = slice(t * BLOCK, min((t + 1) * BLOCK, case["k"]))
                part = s["a"][lo:hi, kk].double() @ b[:, kk].double().t()
                part *= s["sa"][lo:hi, t].double()[:, None]
                c[lo:hi] += part * sb[nrow, t].double()[None, :]
        return {"c": c}
    off = s["offsets"].tolist()
    if kind == "wgrad":
        dw = torch.zeros((case["experts"], case["k"], case["n"]), dtype=torch.float64,
                         device="cuda")
        for e in range(case["experts"]):
            r = slice(off[e], off[e + 1])
            dw[e] = s["a"][r].double().t() @ s["dc"][r].double()
        return {"dw": dw}
    rows, width = (s["dc"], case["k"]) if kind == "dgrad" else (s["a"], case["n"])
    c = torch.zeros((case["tokens"], width), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        r = slice(off[e], off[e + 1])
        w = s["w"][e].double()
        c[r] = rows[r].double() @ (w.t() if kind == "dgrad" else w)
    return {"da" if kind == "dgrad" else "c": c}
