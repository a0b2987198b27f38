"""The operators of a gated recurrent layer on real work: the RMS norm with the
residual's addition (and an 8-bit output with scales), the matrix product with
bias, activation and residual in its epilogue, and the gated linear recurrence,
each forward and backward and in its form for single tokens.

``run`` computes them in a plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where ``own`` is true, by the package's calls;
``exact`` gives the same outputs from the definitions in 64 bits.

    norm        s = x + r;  rstd = (mean s^2 + eps)^(-1/2);  y = s rstd w
                8 bits: scale = max|y| / 448 of the row, q = e4m3(y / scale)
    product     p = (x w^T) sx sw + bias;  y = act(p) + residual
    recurrence  f = sigmoid(g);  h_t = f_t h_{t-1} + (1 - f_t) x_t;  y = h silu(z)
"""
import math

import torch

own = False

BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "f32": F32, "fp8": FP8}
SIZE = {"bf16": 2, "f32": 4, "fp8": 1}
EPS = 1e-5
EVERY = 64           # the recurrence's backward pass starts from the state before every 64th token
E4M3_MAX = 448.0


def listed():
    return [
        # the norm of 16 sequences' next token in the 2.7B-shaped layer, residual stream in 32 bits
        {"name": "norm_decode", "op": "norm_fwd", "rows": 16, "width": 2560, "dtype": "bf16", "residual": "f32", "out": "bf16"},
        # a long prompt through the same layer, its output in 8 bits for an 8-bit product
        {"name": "norm_long_fp8", "op": "norm_fwd", "rows": 65536, "width": 2560, "dtype": "bf16", "residual": "bf16", "out": "fp8"},
        # training at the 370M shape: 8 sequences of 2048 tokens, less the last token of each
        {"name": "norm_train_bwd", "op": "norm_bwd", "rows": 8 * 2047, "width": 1024, "dtype": "bf16", "residual": "f32", "out": "bf16"},
        # one token through the three-in-one input projection of the 2.7B-shaped layer
        {"name": "product_one_token", "op": "linear_fwd", "tokens": 1, "features": 15360, "inner": 2560, "dtype": "bf16", "act": "none", "bias": True, "residual": False},
        # 16 sequences' next token through the output projection, 8-bit weights and activations
        {"name": "product_decode_fp8", "op": "linear_fwd", "tokens": 16, "features": 2560, "inner": 5120, "dtype": "fp8", "act": "none", "bias": False, "residual": True},
        # a prompt of odd length through the 130M shape's expanding product, in 8 bits
        {"name": "product_prompt_fp8", "op": "linear_fwd", "tokens": 4001, "features": 1536, "inner": 768, "dtype": "fp8", "act": "silu", "bias": True, "residual": False},
        # a long prompt through the 2.7B shape's output projection, the residual added in the epilogue
        {"name": "product_long", "op": "linear_fwd", "tokens": 65536, "features": 2560, "inner": 5120, "dtype": "bf16", "act": "silu", "bias": True, "residual": True},
        # the gradients of the 370M shape's expanding product over one training batch
        {"name": "product_train_bwd", "op": "linear_bwd", "tokens": 8 * 2047, "features": 2048, "inner": 1024, "dtype": "bf16", "act": "gelu", "bias": True, "residual": False},
        # one token of 64 layers' recurrences at the 2.7B shape, four sequences
        {"name": "recurrence_step", "op": "scan_step", "rows": 256, "width": 5120, "dtype": "bf16", "gate": True},
        # the recurrence over one long prompt at the 2.7B shape
        {"name": "recurrence_long", "op": "scan_fwd", "seqs": 1, "length": 65536, "packed": False, "width": 5120, "dtype": "bf16", "gate": True},
        # 47 sequences of many lengths laid end to end, in 32 bits, without an output gate
        {"name": "recurrence_packed", "op": "scan_fwd", "seqs": 47, "length": 1394, "packed": True, "width": 1536, "dtype": "f32", "gate": False},
        # the recurrence's gradients in training at the 370M shape
        {"name": "recurrence_train_bwd", "op": "scan_bwd", "seqs": 8, "length": 2047, "packed": False, "width": 2048, "dtype": "bf16", "gate": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _tokens(rng, lo, hi):
    """Any whole number, over its logarithm."""
    n = _log_int(rng, lo, hi)
    return n + 1 if n == 3072 else n


def _width(rng, lo, hi, step):
    """A layer's width: a multiple of `step`, over its logarithm."""
    n = max(lo, _log_int(rng, lo, hi) // step * step)
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "linear_fwd", "linear_fwd", "linear_bwd", "scan_step", "scan_fwd", "scan_fwd", "scan_bwd"])
    if op in ("norm_fwd", "norm_bwd"):
        # widths are multiples of 8, one in four any number
        width = _width(rng, 256, 8192, 8) if rng.random() < 0.75 else _tokens(rng, 256, 8192)
        rows = _tokens(rng, 1, 65536)
        while rows * width > 65536 * 2560:
            rows //= 2
        dtype = rng.choice(["bf16", "bf16", "f32"])
        residual = rng.choice(["none", dtype, "f32"])
        return {"op": op, "rows": rows + (rows == 3072), "width": width, "dtype": dtype, "residual": residual,
                "out": rng.choice([dtype, dtype, "fp8"]) if op == "norm_fwd" else dtype}
    if op in ("linear_fwd", "linear_bwd"):
        features, inner = _width(rng, 256, 16384, 16), _width(rng, 256, 8192, 16)
        tokens = _tokens(rng, 1, 65536) if op == "linear_fwd" else _tokens(rng, 64, 32768)
        most = 65536 * 2560 * 5120 // (1 if op == "linear_fwd" else 3)
        while tokens * features * inner > most or tokens * features > 65536 * 5120:
            tokens //= 2
        return {"op": op, "tokens": tokens + (tokens == 3072), "features": features, "inner": inner,
                "dtype": rng.choice(["bf16", "fp8"]) if op == "linear_fwd" else "bf16",
                "act": rng.choice(["none", "silu", "gelu", "relu"]), "bias": rng.random() < 0.5,
                "residual": op == "linear_fwd" and rng.random() < 0.5}
    if op == "scan_step":
        return {"op": op, "rows": _tokens(rng, 1, 1024), "width": _width(rng, 256, 8192, 2), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "gate": rng.random() < 0.7}
    width = _width(rng, 256, 8192, 2)
    length = _tokens(rng, 1, 65536)
    seqs = rng.randint(1, 64)
    most = 65536 * 5120 // (1 if op == "scan_fwd" else 4)
    while seqs * length * width > most:
        if seqs > 1:
            seqs = seqs // 2
        else:
            length //= 2
    return {"op": op, "seqs": seqs, "length": length + (length == 3072), "packed": rng.random() < 0.4, "width": width,
            "dtype": rng.choice(["bf16", "bf16", "f32"]), "gate": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype, mean=0.0, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen).to(dtype)


def _rows_in_8_bits(t):
    """A float matrix as e4m3 values and one scale a row."""
    amax = t.abs().amax(dim=-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (t / scale[:, None]).to(FP8), scale


def _offsets(case, seed):
    """Sequence offsets on the token axis: all of one length, or, packed, of
    lengths spread over their logarithm with the same sum (some are empty)."""
    n, length = case["seqs"], case["length"]
    if not case["packed"]:
        return [length * i for i in range(n + 1)]
    gen = torch.Generator().manual_seed(seed + 991)
    share = torch.exp(torch.rand(n, generator=gen, dtype=torch.float64) * 5.0)
    cu = torch.cumsum(share, 0) / share.sum() * (n * length)
    return [0] + [int(v) for v in cu[:-1]] + [n * length]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    dt = DTYPES[case["dtype"]]
    if op in ("norm_fwd", "norm_bwd"):
        rows, width = case["rows"], case["width"]
        s["weight"] = _normal(gen, (width,), F32, 1.0, 0.2)
        # rows of a residual stream differ in size, and a few channels are large
        size = torch.exp(_normal(gen, (rows, 1), F32, 0.0, 0.5))
        channel = torch.exp(_normal(gen, (width,), F32, 0.0, 0.5))
        if op == "norm_fwd":
            s["x"] = _normal(gen, (rows, width), dt)
            s["r"] = None if case["residual"] == "none" else (_normal(gen, (rows, width), F32) * size * channel).to(DTYPES[case["residual"]])
        else:
            stream = case["dtype"] if case["residual"] == "none" else case["residual"]
            s["s"] = (_normal(gen, (rows, width), F32) * size * channel).to(DTYPES[stream])
            s["rstd"] = torch.rsqrt(s["s"].float().square().mean(dim=-1) + EPS)
            s["dy"] = _normal(gen, (rows, width), dt)
            s["ds"] = None if case["residual"] == "none" else _normal(gen, (rows, width), s["s"].dtype)
        return s
    if op in ("linear_fwd", "linear_bwd"):
        m, n, k = case["tokens"], case["features"], case["inner"]
        x, w = _normal(gen, (m, k), F32), _normal(gen, (n, k), F32, 0.0, k ** -0.5)
        if case["dtype"] == "fp8":
            (s["x"], s["x_scale"]), (s["w"], s["w_scale"]) = _rows_in_8_bits(x), _rows_in_8_bits(w)
        else:
            s["x"], s["w"], s["x_scale"], s["w_scale"] = x.to(dt), w.to(dt), None, None
        s["bias"] = _normal(gen, (n,), F32, 0.0, 0.5) if case["bias"] else None
        s["residual"] = _normal(gen, (m, n), BF16) if case["residual"] else None
        if op == "linear_bwd":
            s["dy"] = _normal(gen, (m, n), dt)
            # what the forward pass kept: the values before the activation
            s["preact"] = _normal(gen, (m, n), dt) if case["act"] != "none" else None
        return s
    if op == "scan_step":
        shape = (case["rows"], case["width"])
        s["state"] = _normal(gen, shape, F32, 0.0, 0.5)
        s["x"], s["g"] = _normal(gen, shape, dt), _normal(gen, shape, dt, 2.0, 2.0)
        s["z"] = _normal(gen, shape, dt) if case["gate"] else None
        return s
    cu = _offsets(case, seed)
    shape = (cu[-1], case["width"])
    # x, g and z are the parts of one projection's rows, as a layer has them
    parts = 3 if case["gate"] else 2
    rows = torch.empty((shape[0], parts * shape[1]), dtype=dt, device="cuda")
    rows[:, :shape[1]] = _normal(gen, shape, dt)
    rows[:, shape[1]:2 * shape[1]] = _normal(gen, shape, dt, 2.0, 2.0)
    if case["gate"]:
        rows[:, 2 * shape[1]:] = _normal(gen, shape, dt)
    cut = rows if case["packed"] else rows.view(case["seqs"], case["length"], -1)
    width = shape[1]
    s["x"], s["g"], s["z"] = cut[..., :width], cut[..., width:2 * width], cut[..., 2 * width:] if case["gate"] else None
    s["init"] = _normal(gen, (case["seqs"], width), F32, 0.0, 0.5)
    s["cu"], s["cu_dev"] = cu, torch.tensor(cu, dtype=torch.int32, device="cuda")
    if op == "scan_bwd":
        s["dy"] = _normal(gen, tuple(s["x"].shape), dt)
        s["dfinal"] = _normal(gen, (case["seqs"], width), F32)
        # what the forward pass kept: the state before every 64th token
        starts, at, _ = _marks(cu)
        f, u, first = _gates(_flat(s["x"]), _flat(s["g"]), s["init"], starts, at)
        h = _forward(f, u, _longest(cu))
        kept = torch.arange(0, shape[0], EVERY, device="cuda")
        before = torch.cat([torch.zeros((1, width), device="cuda"), h])[kept]
        s["checkpoints"] = torch.where(starts[kept][:, None], first[kept], before)
    return s


# ------------------------------------------------------------- plain forms
def _act(p, name):
    if name == "silu":
        return p / (1 + torch.exp(-p))
    if name == "gelu":
        return 0.5 * p * (1 + torch.erf(p * 0.5 ** 0.5))
    return torch.clamp(p, min=0) if name == "relu" else p


def _act_slope(p, name):
    if name == "silu":
        sig = 1 / (1 + torch.exp(-p))
        return sig * (1 + p * (1 - sig))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(p * 0.5 ** 0.5)) + p * torch.exp(-0.5 * p * p) * (2 * math.pi) ** -0.5
    return (p > 0).to(p.dtype)


def _flat(t):
    return t.reshape(-1, t.shape[-1])


def _longest(cu):
    return max(b - a for a, b in zip(cu, cu[1:]))


def _marks(cu):
    """Per token: whether it begins a sequence, its sequence, and per sequence its last token (-1: empty)."""
    n, total = len(cu) - 1, cu[-1]
    c = torch.tensor(cu, device="cuda")
    at = torch.searchsorted(c, torch.arange(total, device="cuda"), right=True) - 1
    full = c[1:] > c[:-1]
    starts = torch.zeros(total, dtype=torch.bool, device="cuda")
    starts[c[:-1][full]] = True
    return starts, at, torch.where(full, c[1:] - 1, torch.full((n,), -1, device="cuda"))


def _gates(x, g, init, starts, at):
    """f, u with h = f h + u, where a first token has its initial state in u (and f = 0); and the state before each first token."""
    x, g = x.float(), g.float()
    f = 1 / (1 + torch.exp(-g))
    u = x / (1 + torch.exp(g))
    where = starts.nonzero()[:, 0]
    first = torch.zeros_like(x)
    first[where] = init[at[where]]
    u[where] += f[where] * first[where]
    f[where] = 0
    return f, u, first


def _forward(f, u, longest):
    """All h_t = f_t h_{t-1} + u_t, the reach of every value doubled in each step."""
    a, h, d = f.clone(), u.clone(), 1
    while d < longest:
        h[d:] += a[d:] * h[:-d].clone()
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return h


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op == "norm_fwd":
        t = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        rstd = 1 / torch.sqrt((t * t).mean(dim=-1) + EPS)
        y = t * rstd[:, None] * s["weight"]
        out = {"rstd": rstd}
        if s["r"] is not None:
            out["stream"] = t.to(s["r"].dtype)
        if case["out"] == "fp8":
            out["y"], out["scale"] = _rows_in_8_bits(y)
        else:
            out["y"] = y.to(DTYPES[case["out"]])
        return out
    if op == "norm_bwd":
        dy, t, rstd = s["dy"].float() * s["weight"], s["s"].float(), s["rstd"][:, None]
        ds = rstd * (dy - t * rstd * (dy * t * rstd).mean(dim=-1, keepdim=True))
        if s["ds"] is not None:
            ds = ds + s["ds"].float()
        out = {"dx": ds.to(dt), "dweight": (s["dy"].float() * t * rstd).sum(dim=0)}
        if s["s"].dtype != dt:
            out["dstream"] = ds.to(s["s"].dtype)
        return out
    if op == "linear_fwd":
        x, w = s["x"].float(), s["w"].float()
        p = x @ w.t()
        if s["x_scale"] is not None:
            p = p * s["x_scale"][:, None] * s["w_scale"]
        if s["bias"] is not None:
            p = p + s["bias"]
        p = _act(p, case["act"])
        if s["residual"] is not None:
            p = p + s["residual"].float()
        return {"y": p.to(BF16)}
    if op == "linear_bwd":
        dp = s["dy"].float()
        if s["preact"] is not None:
            dp = dp * _act_slope(s["preact"].float(), case["act"])
        out = {"dx": (dp @ s["w"].float()).to(dt), "dw": (dp.t() @ s["x"].float()).to(dt)}
        if s["bias"] is not None:
            out["dbias"] = dp.sum(dim=0)
        return out
    if op == "scan_step":
        g = s["g"].float()
        h = s["state"] / (1 + torch.exp(-g)) + s["x"].float() / (1 + torch.exp(g))
        s["state"].copy_(h)
        if s["z"] is not None:
            h = h * _act(s["z"].float(), "silu")
        return {"y": h.to(dt), "state": s["state"]}
    starts, at, last = _marks(s["cu"])
    x, g = _flat(s["x"]), _flat(s["g"])
    z = None if s["z"] is None else _flat(s["z"]).float()
    f, u, first = _gates(x, g, s["init"], starts, at)
    h = _forward(f, u, _longest(s["cu"]))
    empty = (last < 0)[:, None]
    if op == "scan_fwd":
        final = torch.where(empty, s["init"], h[last])
        return {"y": (h if z is None else h * _act(z, "silu")).to(dt).view(s["x"].shape), "final": final}
    dy = _flat(s["dy"]).float()
    dh = dy if z is None else dy * _act(z, "silu")
    dh = dh.index_add(0, last[~empty[:, 0]], s["dfinal"][~empty[:, 0]])
    # the same recurrence from the last token to the first: lam_t = dh_t + f_{t+1} lam_{t+1}
    back = torch.cat([f[1:], torch.zeros_like(f[:1])]).flip(0)
    lam = _forward(back, dh.flip(0).contiguous(), _longest(s["cu"])).flip(0)
    before = torch.where(starts[:, None], first, torch.cat([torch.zeros_like(h[:1]), h[:-1]]))
    keep, drop = 1 / (1 + torch.exp(-g.float())), 1 / (1 + torch.exp(g.float()))
    dinit = s["dfinal"].clone()
    where = starts.nonzero()[:, 0]
    dinit[at[where]] = (keep * lam)[where]
    out = {"dx": (drop * lam).to(dt).view(s["x"].shape), "dg": (lam * (before - x.float()) * keep * drop).to(dt).view(s["x"].shape), "dinit": dinit}
    if z is not None:
        out["dz"] = (dy * h * _act_slope(z, "silu")).to(dt).view(s["x"].shape)
    return out


# ------------------------------------------------------- the package's calls
def _own(s):
    import state_space_model_chunked_gb300 as ssd
    case, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        y, stream, rstd, scale = ssd.rmsnorm_fwd(s["x"], s["weight"], s["r"], eps=EPS, out_dtype=DTYPES[case["out"]])
        out = {"y": y, "rstd": rstd}
        if stream is not None:
            out["stream"] = stream
        if scale is not None:
            out["scale"] = scale
        return out
    if op == "norm_bwd":
        dx, dstream, dweight = ssd.rmsnorm_bwd(s["dy"], s["s"], s["weight"], s["rstd"], s["ds"])
        out = {"dx": dx, "dweight": dweight}
        if dstream is not dx:
            out["dstream"] = dstream
        return out
    if op == "linear_fwd":
        return {"y": ssd.linear_fwd(s["x"], s["w"], s["bias"], s["residual"], activation=case["act"], x_scale=s["x_scale"], w_scale=s["w_scale"])}
    if op == "linear_bwd":
        dx, dw, dbias = ssd.linear_bwd(s["dy"], s["x"], s["w"], s["preact"], activation=case["act"], bias=s["bias"] is not None)
        out = {"dx": dx, "dw": dw}
        if dbias is not None:
            out["dbias"] = dbias
        return out
    if op == "scan_step":
        return {"y": ssd.gated_state_update(s["state"], s["x"], s["g"], s["z"]), "state": s["state"]}
    packed = {"cu_seqlens": s["cu"], "cu_seqlens_dev": s["cu_dev"]} if case["packed"] else {}
    if op == "scan_fwd":
        y, final = ssd.gated_scan_fwd(s["x"], s["g"], s["z"], s["init"], **packed)
        return {"y": y, "final": final}
    dx, dg, dz, dinit = ssd.gated_scan_bwd(s["dy"], s["x"], s["g"], s["checkpoints"], s["z"], s["init"], s["dfinal"], **packed)
    out = {"dx": dx, "dg": dg, "dinit": dinit}
    if dz is not None:
        out["dz"] = dz
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op in ("norm_fwd", "norm_bwd"):
        n = case["rows"] * case["width"]
        r = SIZE.get(case["residual"], 0)
        if op == "norm_fwd":
            per = b + 2 * r + SIZE[case["out"]]
            extra = 4 * case["width"] + 4 * case["rows"] * (2 if case["out"] == "fp8" else 1)
            return {"bytes": n * per + extra, "flops": 6 * n}
        stream = r or b
        per = b + stream + r + b + (stream if stream != b else 0)
        return {"bytes": n * per + 8 * case["width"] + 4 * case["rows"], "flops": 9 * n}
    if op in ("linear_fwd", "linear_bwd"):
        m, n, k = case["tokens"], case["features"], case["inner"]
        if op == "linear_fwd":
            scales = 4 * (m + n) if case["dtype"] == "fp8" else 0
            return {"bytes": b * (m * k + n * k) + 2 * m * n * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0) + scales, "flops": 2 * m * n * k}
        act = b * m * n if case["act"] != "none" else 0
        return {"bytes": b * (m * n + m * k + n * k) + act + b * (m * k + n * k) + (4 * n if case["bias"] else 0), "flops": 4 * m * n * k}
    if op == "scan_step":
        n = case["rows"] * case["width"]
        return {"bytes": n * (8 + b * (4 if case["gate"] else 3)), "flops": n * (20 if case["gate"] else 12)}
    n, ends = case["seqs"] * case["length"] * case["width"], 4 * case["seqs"] * case["width"]
    if op == "scan_fwd":
        return {"bytes": n * b * (4 if case["gate"] else 3) + 2 * ends, "flops": n * (20 if case["gate"] else 12)}
    kept = 4 * -(-case["seqs"] * case["length"] // EVERY) * case["width"]
    return {"bytes": n * b * (7 if case["gate"] else 5) + kept + 3 * ends, "flops": n * (40 if case["gate"] else 24)}


# ------------------------------------------------------------------- exact
def _sigmoid64(t):
    return torch.sigmoid(t.double())


def _exact_act(p, name):
    if name == "silu":
        return p * torch.sigmoid(p)
    if name == "gelu":
        return p * 0.5 * torch.erfc(-p / math.sqrt(2.0))
    return p * (p > 0) if name == "relu" else p


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        t = s["x"].double()
        if s["r"] is not None:
            t += s["r"].double()
        rms = torch.sqrt(torch.linalg.vector_norm(t, dim=1) ** 2 / case["width"] + EPS)
        y = t / rms[:, None] * s["weight"].double()
        out = {"rstd": 1 / rms, "y": y}
        if s["r"] is not None:
            out["stream"] = t
        if case["out"] == "fp8":
            top = y.abs().amax(dim=1)
            out["scale"] = torch.where(top > 0, top / E4M3_MAX, 1.0)
            out["y"] = (y / out["scale"][:, None])
        return out
    if op == "norm_bwd":
        # through the unit vectors: y = w v sqrt-mean; the projection of the gradient off the row's direction
        t, rstd = s["s"].double(), s["rstd"].double()[:, None]
        v = t * rstd
        e = s["dy"].double() * s["weight"].double()
        ds = (e - v * ((e * v).sum(dim=1, keepdim=True) / case["width"])) * rstd
        if s["ds"] is not None:
            ds += s["ds"].double()
        out = {"dx": ds, "dweight": torch.einsum("rc,rc->c", s["dy"].double(), v)}
        if s["s"].dtype != DTYPES[case["dtype"]]:
            out["dstream"] = ds
        return out
    if op == "linear_fwd":
        if case["tokens"] * case["features"] * case["inner"] > 1 << 42:
            return None
        x, w = s["x"].float().double(), s["w"].float().double()
        if s["x_scale"] is not None:
            x, w = x * s["x_scale"].double()[:, None], w * s["w_scale"].double()[:, None]
        p = torch.einsum("mk,nk->mn", x, w)
        if s["bias"] is not None:
            p += s["bias"].double()
        p = _exact_act(p, case["act"])
        return {"y": p if s["residual"] is None else p + s["residual"].double()}
    if op == "linear_bwd":
        dp = s["dy"].double()
        if s["preact"] is not None:
            p = s["preact"].double().requires_grad_(True)
            _exact_act(p, case["act"]).backward(dp)
            dp = p.grad
        out = {"dx": torch.einsum("mn,nk->mk", dp, s["w"].double()), "dw": torch.einsum("mn,mk->nk", dp, s["x"].double())}
        if s["bias"] is not None:
            out["dbias"] = dp.sum(dim=0)
        return out
    if op == "scan_step":
        f = _sigmoid64(s["g"])
        h = f * s["state"].double() + _sigmoid64(-s["g"].double()) * s["x"].double()
        return {"y": h if s["z"] is None else h * _exact_act(s["z"].double(), "silu"), "state": h}
    # the recurrence, one token after another, all sequences at once
    n, width, cu = case["seqs"], case["width"], s["cu"]
    x, g = s["x"].reshape(-1, width), s["g"].reshape(-1, width)
    total, longest = cu[-1], max(b - a for a, b in zip(cu, cu[1:]))
    if longest > (70000 if op == "scan_fwd" else 40000) or total * width > 1 << 29:
        return None
    order = sorted(range(n), key=lambda i: cu[i] - cu[i + 1])
    lens = [cu[i + 1] - cu[i] for i in order]
    first = torch.tensor([cu[i] for i in order], device="cuda")
    h = s["init"][order].double()
    hs = torch.empty((total, width), dtype=torch.float64, device="cuda")
    live = n
    for t in range(longest):
        while live and lens[live - 1] <= t:
            live -= 1
        if n == 1:
            f, v = torch.sigmoid(g[t:t + 1].double()), x[t:t + 1].double()
            h = v + f * (h - v)
            hs[t] = h[0]
        else:
            rows = first[:live] + t
            f, v = torch.sigmoid(g[rows].double()), x[rows].double()
            h[:live] = v + f * (h[:live] - v)
            hs[rows] = h[:live]
    z = None if s["z"] is None else s["z"].reshape(-1, width).double()
    shape = s["x"].shape
    if op == "scan_fwd":
        final = torch.empty_like(h)
        final[order] = h
        return {"y": (hs if z is None else hs * _exact_act(z, "silu")).view(shape), "final": final}
    dy = s["dy"].reshape(-1, width).double()
    sig = None if z is None else torch.sigmoid(z)
    dh = dy if z is None else dy * z * sig
    lam = s["dfinal"][order].double()
    dx, dg = torch.empty_like(hs), torch.empty_like(hs)
    init = s["init"][order].double()
    for t in range(longest - 1, -1, -1):
        while live < n and lens[live] > t:
            live += 1
        rows = first[:live] + t
        f, v = torch.sigmoid(g[rows].double()), x[rows].double()
        before = init[:live] if t == 0 else hs[rows - 1]
        total_grad = lam[:live] + dh[rows]
        dx[rows] = total_grad * torch.sigmoid(-g[rows].double())
        dg[rows] = total_grad * (before - v) * f * torch.sigmoid(-g[rows].double())
        lam[:live] = total_grad * f
    dinit = torch.empty_like(lam)
    dinit[order] = lam
    out = {"dx": dx.view(shape), "dg": dg.view(shape), "dinit": dinit}
    if z is not None:
        out["dz"] = (dy * hs * sig * (1 + z * (1 - sig))).view(shape)
    return out
