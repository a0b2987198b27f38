"""The operators of a delta-rule language model on real work: the embedding's
lookup and its gradient, the layer norm with the residual's addition, and the gated
delta rule over sequences, each forward and backward, and the delta rule's single
token.

``run`` computes them in a plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where ``own`` is true, by the package's calls;
``exact`` gives the same outputs from the definitions in 64 bits.

    embedding   y = table[token] scale; a token outside the table is padding: a row of zeros
                dtable[v] = scale * the sum of dy over the tokens that are v
    layer norm  s = x + r;  y = (s - mean) rstd w + bias;  rstd = (mean (s - mean)^2 + eps)^(-1/2)
                8 bits: scale = max|y| / 448 of the row, q = e4m3(y / scale)
    delta rule  S' = exp(g_t) S_{t-1};  u = beta_t (v_t - S' k_t);  S_t = S' + u k_t^T
                o_t = scale S_t q_t          S [P][N] a head; q, k shared by heads of a group
"""
import math

import torch

own = False

BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "f32": F32, "fp8": FP8}
SIZE = {"bf16": 2, "f32": 4, "fp8": 1}
EPS = 1e-5
EVERY = 64           # the delta rule's backward pass starts from the state before every 64th token of a sequence
E4M3_MAX = 448.0
DEVICE = "cuda"


def listed():
    return [
        # 16 sequences' next token looked up for the 2.7B-shaped layer's residual stream in 32 bits
        {"name": "embedding_decode", "op": "embed_fwd", "seqs": 16, "length": 1, "vocab": 50000, "width": 2560, "dtype": "bf16", "out": "f32", "padded": False},
        # a long prompt's rows, as they lie in the table
        {"name": "embedding_long", "op": "embed_fwd", "seqs": 1, "length": 65536, "vocab": 50000, "width": 2560, "dtype": "bf16", "out": "bf16", "padded": False},
        # the table's gradient of a training batch at the 370M shape, its sequences padded to one length
        {"name": "embedding_train_bwd", "op": "embed_bwd", "seqs": 8, "length": 2047, "vocab": 50000, "width": 1024, "dtype": "bf16", "out": "f32", "padded": True},
        # the norm of 16 sequences' next token, residual stream in 32 bits
        {"name": "layernorm_decode", "op": "norm_fwd", "rows": 16, "width": 2560, "dtype": "bf16", "residual": "f32", "out": "bf16", "bias": True},
        # a long prompt's norm with its output in 8 bits for an 8-bit product
        {"name": "layernorm_long_fp8", "op": "norm_fwd", "rows": 65536, "width": 2560, "dtype": "bf16", "residual": "bf16", "out": "fp8", "bias": True},
        # training at the 370M shape: 8 sequences of 2048 tokens, less the last token of each
        {"name": "layernorm_train_bwd", "op": "norm_bwd", "rows": 8 * 2047, "width": 1024, "dtype": "bf16", "residual": "f32", "out": "bf16", "bias": True},
        # the next token of 16 sequences through 32 heads
        {"name": "delta_step", "op": "delta_step", "seqs": 16, "length": 1, "heads": 32, "groups": 16, "p": 128, "n": 128, "dtype": "bf16", "packed": False},
        # four short prompts through a small layer in 32 bits
        {"name": "delta_short_f32", "op": "delta_fwd", "seqs": 4, "length": 77, "heads": 8, "groups": 8, "p": 64, "n": 64, "dtype": "f32", "packed": False},
        # one long prompt
        {"name": "delta_long", "op": "delta_fwd", "seqs": 1, "length": 65536, "heads": 32, "groups": 16, "p": 128, "n": 128, "dtype": "bf16", "packed": False},
        # 47 sequences of many lengths laid end to end, the 130M shape's heads of 64 channels by 128 state columns
        {"name": "delta_packed", "op": "delta_fwd", "seqs": 47, "length": 1394, "heads": 24, "groups": 1, "p": 64, "n": 128, "dtype": "bf16", "packed": True},
        # the gradients of a training batch
        {"name": "delta_train_bwd", "op": "delta_bwd", "seqs": 8, "length": 2047, "heads": 16, "groups": 16, "p": 128, "n": 128, "dtype": "bf16", "packed": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "delta_step", "delta_fwd", "delta_fwd", "delta_bwd"])
    # widths are multiples of 8, one in four any number
    width = _log_int(rng, 256, 8192) // 8 * 8 if rng.random() < 0.75 else _log_int(rng, 256, 8192)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("embed_fwd", "embed_bwd"):
        vocab, seqs, length = _log_int(rng, 256, 250000), rng.randint(1, 64), _log_int(rng, 1, 65536)
        while seqs * length * width > 65536 * 2560 or seqs * length > 65536:
            seqs, length = (seqs // 2, length) if seqs > 1 else (1, length // 2)
        while vocab * width > 50000 * 2560 or (op == "embed_bwd" and vocab * width > 50000 * 1024):
            vocab //= 2
        return {"op": op, "seqs": seqs, "length": length, "vocab": vocab, "width": width, "dtype": dtype,
                "out": rng.choice([dtype, "f32"]), "padded": rng.random() < 0.5}
    if op in ("norm_fwd", "norm_bwd"):
        rows = _log_int(rng, 1, 65536)
        while rows * width > 65536 * 2560:
            rows //= 2
        return {"op": op, "rows": rows, "width": width, "dtype": dtype, "residual": rng.choice(["none", dtype, "f32"]),
                "out": rng.choice([dtype, dtype, "fp8"]) if op == "norm_fwd" else dtype, "bias": rng.random() < 0.7}
    groups = rng.randint(1, 16)
    heads = groups * rng.choice([1, 1, 2, 4])
    p, n = (rng.choice([64, 128]), rng.choice([64, 128])) if rng.random() < 0.75 else (rng.randint(1, 32) * 4, rng.randint(1, 32) * 4)
    case = {"op": op, "seqs": rng.randint(1, 64), "length": 1, "heads": heads, "groups": groups, "p": p, "n": n, "dtype": dtype, "packed": False}
    if op == "delta_step":
        case["seqs"] = _log_int(rng, 1, 512)
        while case["seqs"] * heads * p * n > 1 << 26:
            case["seqs"] //= 2
        return case
    case["length"], case["packed"] = _log_int(rng, 1, 65536), rng.random() < 0.4
    most = (65536 * 32 if op == "delta_fwd" else 8 * 2047 * 16) * 128 * 128
    while (case["seqs"] * case["length"] * heads * p * n > most or case["seqs"] * case["length"] * heads * 128 * 128 > 2 * most
           or case["length"] > (65536 if op == "delta_fwd" else 8192)):
        if case["seqs"] > 1:
            case["seqs"] //= 2
        else:
            case["length"] //= 2
    return case


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype=F32, mean=0.0, std=1.0):
    return torch.empty(shape, dtype=F32, device=DEVICE).normal_(mean, std, generator=gen).to(dtype)


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


def _token_ids(gen, case):
    """Tokens as frequent as words of a text: the r-th most frequent about 1 / r."""
    name = torch.randperm(case["vocab"], generator=gen, device=DEVICE)
    share = torch.rand((case["seqs"], case["length"]), dtype=torch.float64, generator=gen, device=DEVICE)
    rank = 2.7 * torch.expm1(share * math.log1p(case["vocab"] / 2.7))
    ids = name[rank.long().clamp_max(case["vocab"] - 1)]
    if case["padded"]:
        # each sequence ends somewhere in its last quarter
        lens = (case["length"] * (0.75 + 0.25 * torch.rand((case["seqs"], 1), generator=gen, device=DEVICE))).ceil()
        ids = torch.where(torch.arange(case["length"], device=DEVICE) < lens, ids, torch.full_like(ids, -1))
    return ids


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, s = case["op"], {"case": case}
    dt = DTYPES[case["dtype"]]
    if op in ("embed_fwd", "embed_bwd"):
        s["tokens"] = _token_ids(gen, case)
        s["scale"] = case["width"] ** 0.5
        if op == "embed_fwd":
            s["table"] = _normal(gen, (case["vocab"], case["width"]), dt, 0.0, 0.02)
        else:
            s["dy"] = _normal(gen, (case["seqs"], case["length"], case["width"]), dt)
        return s
    if op in ("norm_fwd", "norm_bwd"):
        rows, width = case["rows"], case["width"]
        s["weight"] = _normal(gen, (width,), F32, 1.0, 0.2)
        s["bias"] = _normal(gen, (width,), F32, 0.0, 0.2) if case["bias"] else None
        # rows of a residual stream differ in size, a few channels are large, and the mean is not zero
        size = torch.exp(_normal(gen, (rows, 1), F32, 0.0, 0.5))
        channel = torch.exp(_normal(gen, (width,), F32, 0.0, 0.5))
        stream = (_normal(gen, (rows, width), F32, 0.3) * size * channel).to(dt if case["residual"] == "none" else DTYPES[case["residual"]])
        if op == "norm_fwd":
            s["r"] = None if case["residual"] == "none" else stream
            s["x"] = stream if case["residual"] == "none" else _normal(gen, (rows, width), dt)
        else:
            s["s"] = stream
            wide = stream.double()
            s["mean"] = wide.mean(dim=-1).float()
            s["rstd"] = torch.rsqrt(wide.var(dim=-1, unbiased=False) + EPS).float()
            s["dy"] = _normal(gen, (rows, width), dt)
            s["ds"] = None if case["residual"] == "none" else _normal(gen, (rows, width), stream.dtype)
        return s
    heads, groups, p, n = case["heads"], case["groups"], case["p"], case["n"]
    cu = _offsets(case, seed)
    total = cu[-1]
    # q and k are activated and normalized, as a layer hands them over
    q, k = (torch.nn.functional.silu(_normal(gen, (total, groups, n), F32, 0.0, 2.0)) for _ in range(2))
    q, k = ((t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dt) for t in (q, k))
    v = _normal(gen, (total, heads, p), dt)
    # heads forget at rates spread over a factor of 16
    rate = torch.exp(torch.rand((heads,), generator=gen, device=DEVICE) * math.log(16.0))
    g = -rate * torch.nn.functional.softplus(_normal(gen, (total, heads), F32, -4.0, 1.0))
    beta = torch.sigmoid(_normal(gen, (total, heads)))
    s["scale"] = n ** -0.5
    state = _normal(gen, (case["seqs"], heads, p, n), F32, 0.0, 0.3)
    if op == "delta_step":
        s.update(q=q, k=k, v=v, g=g, beta=beta, state=state, next=torch.empty_like(state))
        return s
    s["cu"], s["cu_dev"], s["init"] = cu, torch.tensor(cu, dtype=torch.int32, device=DEVICE), state
    if op == "delta_bwd":
        s["do"] = _normal(gen, (total, heads, p), dt)
        s["dfinal"] = _normal(gen, (case["seqs"], heads, p, n))
        # what the forward pass kept: the state before every 64th token of each sequence
        x = _padded({"q": q, "k": k, "v": v, "g": g, "beta": beta}, cu, groups, heads)
        _, _, starts = _delta_forward(x, state, s["scale"])
        kept = torch.zeros((total // EVERY + case["seqs"], heads, p, n), device=DEVICE)
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            chunks = -(-(b - a) // EVERY)
            kept[a // EVERY + i:a // EVERY + i + chunks] = starts[:chunks, i]
        s["checkpoints"] = kept
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("do", s.get("do"))):
        if t is not None:
            s[name] = t if case["packed"] else t.view((case["seqs"], case["length"]) + tuple(t.shape[1:]))
    return s


# ------------------------------------------------------------- plain forms
def _flat(t, case):
    return t if case["packed"] else t.reshape((-1,) + tuple(t.shape[2:]))


def _places(cu):
    """Of every token its sequence and its place in it."""
    c = torch.tensor(cu, device=DEVICE)
    t = torch.arange(cu[-1], device=DEVICE)
    seq = torch.searchsorted(c, t, right=True) - 1
    return seq, t - c[seq]


def _padded(parts, cu, groups, heads):
    """The parts' tokens as [chunk][sequence][head][place][...] in 32 bits, zeros behind each sequence."""
    seq, place = _places(cu)
    chunks = max(1, -(-max(b - a for a, b in zip(cu, cu[1:])) // EVERY))
    out = {}
    for name, t in parts.items():
        t = t.float()
        if t.shape[1] == groups and t.dim() == 3 and name in ("q", "k"):
            t = t.repeat_interleave(heads // groups, dim=1)
        pad = torch.zeros((chunks * EVERY, len(cu) - 1) + tuple(t.shape[1:]), device=DEVICE)
        pad[place, seq] = t
        pad = pad.view((chunks, EVERY) + tuple(pad.shape[1:]))
        out[name] = pad.permute(0, 2, 3, 1, *range(4, pad.dim()))
    return out


def _tokens_of(t, cu):
    """_padded's order back to tokens."""
    seq, place = _places(cu)
    t = t.permute(0, 3, 1, 2, *range(4, t.dim()))
    return t.reshape((-1,) + tuple(t.shape[2:]))[place, seq]


def _chunk_terms(x, scale):
    """Of all chunks: the decays from the chunk's start (up to each token, and the whole), to its end,
    between tokens, the products of keys and of queries with keys, and the inverse of the unit triangle."""
    sums = torch.cumsum(x["g"].double(), dim=-1)
    lower = torch.ones((EVERY, EVERY), dtype=torch.bool, device=DEVICE).tril()
    between = torch.exp(torch.where(lower, sums[..., :, None] - sums[..., None, :], -math.inf)).float()
    upto, toend = torch.exp(sums).float()[..., None], torch.exp(sums[..., -1:] - sums).float()[..., None]
    kk = x["k"] @ x["k"].mT * between
    qk = x["q"] @ x["k"].mT * between * scale
    a = -(x["beta"][..., None] * kk).tril(-1)
    inverse = torch.eye(EVERY, device=DEVICE) + a
    for _ in range(5):      # (1 - a)^-1 = (1 + a)(1 + a^2)(1 + a^4) ... : a^64 is zero
        a = a @ a
        inverse = inverse + inverse @ a
    return upto, toend, between, kk, qk, inverse


def _delta_forward(x, state, scale):
    """(o, the last state, the state before every chunk) of _padded's parts."""
    upto, toend, _, _, qk, inverse = _chunk_terms(x, scale)
    state, starts, outs = state.mT, [], []
    for c in range(x["q"].shape[0]):
        starts.append(state.mT)
        r = x["v"][c] - upto[c] * (x["k"][c] @ state)
        u = inverse[c] @ (x["beta"][c][..., None] * r)
        outs.append(scale * upto[c] * (x["q"][c] @ state) + qk[c] @ u)
        state = upto[c][..., -1:, :] * state + x["k"][c].mT @ (toend[c] * u)
    return torch.stack(outs), state.mT, torch.stack(starts)


def _delta_backward(x, starts, dstate, scale):
    """The gradients of q, k, v, g, beta (by head) and of the initial state."""
    upto, toend, between, kk, qk, inverse = _chunk_terms(x, scale)
    dstate = dstate.mT
    got = {name: [] for name in ("q", "k", "v", "g", "beta")}
    for c in reversed(range(x["q"].shape[0])):
        q, k, v, do, beta, state = x["q"][c], x["k"][c], x["v"][c], x["do"][c], x["beta"][c][..., None], starts[c].mT
        ks = upto[c] * (k @ state)
        r = v - ks
        u = inverse[c] @ (beta * r)
        kd = toend[c] * (k @ dstate)
        dur = inverse[c].mT @ (qk[c].mT @ do + kd)
        dr = beta * dur
        dqk = (do @ u.mT).tril() * between[c] * scale
        da = -(dur @ u.mT).tril(-1)
        dkk = beta * da * between[c]
        qs = scale * upto[c] * (do @ state.mT)
        ks_grad = -upto[c] * (dr @ state.mT)
        got["q"].append(qs + dqk @ k)
        got["k"].append(ks_grad + toend[c] * (u @ dstate.mT) + dqk.mT @ q + dkk @ k + dkk.mT @ k)
        got["v"].append(dr)
        got["beta"].append((dur * r).sum(dim=-1) + (da * kk[c]).sum(dim=-1))
        # of the sums of g: what a token's own sum weighs, less what is weighed by the sums before it
        e = dqk * (q @ k.mT) + dkk * (k @ k.mT)
        inside = torch.cumsum(e.flip(-2), dim=-2).flip(-2)                  # over the tokens from t on
        inside = torch.cumsum(inside, dim=-1) - inside                      # and those before t
        inside = torch.diagonal(inside, dim1=-2, dim2=-1)
        ahead = (qs * q).sum(dim=-1) + (ks_grad * k).sum(dim=-1)            # tokens from t on read the state before the chunk
        behind = (u * kd).sum(dim=-1)                                       # tokens before t write the one behind it
        whole = (upto[c][..., -1:, :] * state * dstate).sum(dim=(-2, -1))[..., None]
        got["g"].append(inside + torch.cumsum(ahead.flip(-1), -1).flip(-1) + torch.cumsum(behind, -1) - behind + whole)
        dstate = upto[c][..., -1:, :] * dstate + scale * q.mT @ (upto[c] * do) - k.mT @ (upto[c] * dr)
    return {name: torch.stack(t[::-1]) for name, t in got.items()}, dstate.mT


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op == "embed_fwd":
        ids = s["tokens"]
        real = (ids >= 0) & (ids < case["vocab"])
        y = s["table"][torch.where(real, ids, 0)].float() * s["scale"]
        return {"y": torch.where(real[..., None], y, 0.0).to(DTYPES[case["out"]])}
    if op == "embed_bwd":
        ids = s["tokens"].reshape(-1)
        real = (ids >= 0) & (ids < case["vocab"])
        dtable = torch.zeros((case["vocab"] + 1, case["width"]), device=DEVICE)
        dtable.index_add_(0, torch.where(real, ids, case["vocab"]), s["dy"].reshape(-1, case["width"]).float())
        return {"dtable": (dtable[:-1] * s["scale"]).to(DTYPES[case["out"]])}
    if op == "norm_fwd":
        t = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        mean = t.mean(dim=-1)
        away = t - mean[:, None]
        rstd = 1 / torch.sqrt((away * away).mean(dim=-1) + EPS)
        y = away * rstd[:, None] * s["weight"]
        if s["bias"] is not None:
            y = y + s["bias"]
        out = {"mean": mean, "rstd": rstd}
        if s["r"] is not None:
            out["stream"] = t.to(s["r"].dtype)
        if case["out"] == "fp8":
            out["y"], out["scale"] = _rows_in_8_bits(y)
        else:
            out["y"] = y.to(DTYPES[case["out"]])
        return out
    if op == "norm_bwd":
        dy, hat = s["dy"].float(), (s["s"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        e = dy * s["weight"]
        ds = s["rstd"][:, None] * (e - e.mean(dim=-1, keepdim=True) - hat * (e * hat).mean(dim=-1, keepdim=True))
        if s["ds"] is not None:
            ds = ds + s["ds"].float()
        out = {"dx": ds.to(dt), "dweight": (dy * hat).sum(dim=0)}
        if s["bias"] is not None:
            out["dbias"] = dy.sum(dim=0)
        if s["s"].dtype != dt:
            out["dstream"] = ds.to(s["s"].dtype)
        return out
    heads, groups = case["heads"], case["groups"]
    if op == "delta_step":
        q, k = (s[name].float().repeat_interleave(heads // groups, dim=1)[:, :, None, :] for name in ("q", "k"))
        state = s["state"] * torch.exp(s["g"])[..., None, None]
        u = s["beta"][..., None] * (s["v"].float() - (state * k).sum(dim=-1))
        state = state + u[..., None] * k
        s["next"].copy_(state)
        return {"o": (s["scale"] * (state * q).sum(dim=-1)).to(dt), "state": s["next"]}
    cu = s["cu"]
    x = _padded({name: _flat(s[name], case) for name in ("q", "k", "v", "g", "beta", "do") if name in s}, cu, groups, heads)
    if op == "delta_fwd":
        o, final, _ = _delta_forward(x, s["init"], s["scale"])
        return {"o": _tokens_of(o, cu).to(dt).view(s["v"].shape), "final": final}
    starts = torch.zeros((x["q"].shape[0],) + tuple(s["dfinal"].shape), device=DEVICE)
    at, last = torch.tensor(cu, device=DEVICE), torch.arange(case["seqs"], device=DEVICE)
    chunks = (at[1:] - at[:-1] + EVERY - 1) // EVERY
    c = torch.arange(x["q"].shape[0], device=DEVICE)[:, None]
    live = c < chunks
    starts[live] = s["checkpoints"][(at[:-1] // EVERY + last + c)[live]]
    grads, dinit = _delta_backward(x, starts, s["dfinal"], s["scale"])
    out = {"dinit": dinit}
    for name, t in grads.items():
        t = _tokens_of(t, cu)
        if name in ("q", "k"):
            t = t.view(t.shape[0], groups, heads // groups, -1).sum(dim=2)
        out["d" + name] = t.to(s[name].dtype).view(s[name].shape)
    return out


# ------------------------------------------------------- the package's calls
def _own(s):
    import state_space_model_chunked_gb300 as ssd
    case, op = s["case"], s["case"]["op"]
    if op == "embed_fwd":
        return {"y": ssd.embedding_fwd(s["tokens"], s["table"], scale=s["scale"], out_dtype=DTYPES[case["out"]])}
    if op == "embed_bwd":
        return {"dtable": ssd.embedding_bwd(s["dy"], s["tokens"], case["vocab"], scale=s["scale"], dtype=DTYPES[case["out"]])}
    if op == "norm_fwd":
        y, stream, mean, rstd, scale = ssd.layernorm_fwd(s["x"], s["weight"], s["bias"], s["r"], eps=EPS, out_dtype=DTYPES[case["out"]])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if stream is not None:
            out["stream"] = stream
        if scale is not None:
            out["scale"] = scale
        return out
    if op == "norm_bwd":
        dx, dstream, dweight, dbias = ssd.layernorm_bwd(s["dy"], s["s"], s["weight"], s["mean"], s["rstd"], s["ds"], bias=s["bias"] is not None)
        out = {"dx": dx, "dweight": dweight}
        if dbias is not None:
            out["dbias"] = dbias
        if dstream is not dx:
            out["dstream"] = dstream
        return out
    if op == "delta_step":
        o = ssd.delta_state_update(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], state_out=s["next"])
        return {"o": o, "state": s["next"]}
    packed = {"cu_seqlens": s["cu"], "cu_seqlens_dev": s["cu_dev"]} if case["packed"] else {}
    if op == "delta_fwd":
        o, final = ssd.delta_scan_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["init"], scale=s["scale"], **packed)
        return {"o": o, "final": final}
    got = ssd.delta_scan_bwd(s["do"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["checkpoints"], s["dfinal"], scale=s["scale"], **packed)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), got))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op in ("embed_fwd", "embed_bwd"):
        tokens, out = case["seqs"] * case["length"], SIZE[case["out"]]
        if op == "embed_fwd":
            # a row that occurs again need not be read again
            return {"bytes": 8 * tokens + min(tokens, case["vocab"]) * case["width"] * b + tokens * case["width"] * out, "flops": tokens * case["width"]}
        return {"bytes": 8 * tokens + tokens * case["width"] * b + case["vocab"] * case["width"] * out, "flops": tokens * case["width"]}
    if op in ("norm_fwd", "norm_bwd"):
        n, vectors = case["rows"] * case["width"], (2 if case["bias"] else 1) * 4 * case["width"]
        r = SIZE.get(case["residual"], 0)
        if op == "norm_fwd":
            return {"bytes": n * (b + 2 * r + SIZE[case["out"]]) + vectors + 4 * case["rows"] * (3 if case["out"] == "fp8" else 2), "flops": 9 * n}
        stream = r or b
        per = b + stream + r + b + (stream if stream != b else 0)
        return {"bytes": n * per + 4 * case["width"] + vectors + 8 * case["rows"], "flops": 13 * n}
    tokens, heads, groups, p, n = case["seqs"] * case["length"], case["heads"], case["groups"], case["p"], case["n"]
    states = case["seqs"] * heads * p * n * 4
    rows, gates = tokens * (2 * groups * n + 2 * heads * p) * b, 8 * tokens * heads
    if op in ("delta_step", "delta_fwd"):
        return {"bytes": rows + gates + 2 * states, "flops": 7 * tokens * heads * p * n}
    kept = (tokens // EVERY + 1) * heads * p * n * 4
    return {"bytes": rows + gates + kept + 2 * states + tokens * (2 * groups * n + heads * p) * b + gates, "flops": 20 * tokens * heads * p * n}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        table = torch.cat([s["table"].double() * s["scale"], torch.zeros((1, case["width"]), dtype=torch.float64, device=DEVICE)])
        return {"y": table[s["tokens"]]}
    if op == "embed_bwd":
        # by sorted tokens: differences of running sums at the ends of each token's rows
        ids, order = torch.sort(s["tokens"].reshape(-1), stable=True)
        sums = torch.zeros((ids.numel() + 1, case["width"]), dtype=torch.float64, device=DEVICE)
        torch.cumsum(s["dy"].reshape(-1, case["width"])[order].double(), dim=0, out=sums[1:])
        ends = torch.searchsorted(ids, torch.arange(-1, case["vocab"], device=DEVICE), right=True)
        return {"dtable": (sums[ends[1:]] - sums[ends[:-1]]) * s["scale"]}
    if op == "norm_fwd":
        t = s["x"].double()
        if s["r"] is not None:
            t = t + s["r"].double()
        var, mean = torch.var_mean(t, dim=1, unbiased=False)
        y = torch.addcmul(torch.zeros_like(t) if s["bias"] is None else s["bias"].double().expand_as(t), (t - mean[:, None]) / torch.sqrt(var + EPS)[:, None], s["weight"].double())
        out = {"mean": mean, "rstd": (var + EPS) ** -0.5, "y": y}
        if s["r"] is not None:
            out["stream"] = t
        if case["out"] == "fp8":
            top = y.abs().amax(dim=1)
            out["scale"] = torch.where(top > 0, top / E4M3_MAX, 1.0)
            out["y"] = y / out["scale"][:, None]
        return out
    if op == "norm_bwd":
        # ds is rstd times e without its parts along the constant row and along the normalized one
        rstd = s["rstd"].double()[:, None]
        hat = (s["s"].double() - s["mean"].double()[:, None]) * rstd
        e = s["dy"].double() * s["weight"].double()
        ds = rstd * (e - e.sum(1, keepdim=True) / case["width"] - hat * (torch.einsum("rc,rc->r", e, hat) / case["width"])[:, None])
        if s["ds"] is not None:
            ds = ds + s["ds"].double()
        out = {"dx": ds, "dweight": torch.einsum("rc,rc->c", s["dy"].double(), hat)}
        if s["bias"] is not None:
            out["dbias"] = s["dy"].double().sum(dim=0)
        if s["s"].dtype != DTYPES[case["dtype"]]:
            out["dstream"] = ds
        return out
    # the delta rule, one token after another, all sequences and heads at once
    heads, groups, p, n = case["heads"], case["groups"], case["p"], case["n"]
    if op == "delta_step":
        q, k = (s[name].double().repeat_interleave(heads // groups, dim=1) for name in ("q", "k"))
        state = torch.exp(s["g"].double())[..., None, None] * s["state"].double()
        u = s["beta"].double()[..., None] * (s["v"].double() - torch.einsum("bhpn,bhn->bhp", state, k))
        state = state + torch.einsum("bhp,bhn->bhpn", u, k)
        return {"o": s["scale"] * torch.einsum("bhpn,bhn->bhp", state, q), "state": state}
    cu, seqs = s["cu"], case["seqs"]
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    back = op == "delta_bwd"
    if longest > (70000 if not back else 9000) or longest * seqs * heads * p * n > ((1 << 36) if not back else (3 << 31)) or cu[-1] == 0:
        return None
    q, k, v, g, beta = (_flat(s[name], case) for name in ("q", "k", "v", "g", "beta"))
    order = sorted(range(seqs), key=lambda i: cu[i] - cu[i + 1])
    lens = [cu[i + 1] - cu[i] for i in order]
    first = torch.tensor([cu[i] for i in order], device=DEVICE)
    wide = heads // groups

    def token(rows):
        keys, asks = (t[rows].double().repeat_interleave(wide, dim=1)[..., None] for t in (k, q))
        return asks, keys, v[rows].double()[..., None], torch.exp(g[rows].double())[..., None, None], beta[rows].double()[..., None, None]

    state = s["init"][order].double()
    o = torch.empty((cu[-1], heads, p), dtype=torch.float64, device=DEVICE)
    past, live = [], seqs
    for t in range(longest):
        while live and lens[live - 1] <= t:
            live -= 1
        rows = first[:live] + t
        asks, keys, value, decay, rate = token(rows)
        if back:
            past.append(state[:live].clone())
        faded = state[:live] * decay
        state[:live] = faded + rate * (value - faded @ keys) @ keys.mT
        o[rows] = s["scale"] * (state[:live] @ asks)[..., 0]
    if not back:
        final = torch.empty_like(state)
        final[order] = state
        return {"o": o.view(s["v"].shape), "final": final}
    do, d = _flat(s["do"], case), s["dfinal"][order].double()
    out = {name: torch.empty(tuple(t.shape[:1]) + (heads,) + tuple(t.shape[2:]), dtype=torch.float64, device=DEVICE)
           for name, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    for t in range(longest - 1, -1, -1):
        while live < seqs and lens[live] > t:
            live += 1
        rows = first[:live] + t
        asks, keys, value, decay, rate = token(rows)
        before = past.pop()
        faded = before * decay
        miss = value - faded @ keys
        now = faded + rate * miss @ keys.mT
        dout = s["scale"] * do[rows].double()[..., None]
        dnow = d[:live] + dout @ asks.mT
        dwrite = dnow @ keys                    # of rate * miss
        dfaded = dnow - rate * dwrite @ keys.mT
        out["dq"][rows] = (now.mT @ dout)[..., 0]
        out["dk"][rows] = (dnow.mT @ (rate * miss) - faded.mT @ (rate * dwrite))[..., 0]
        out["dv"][rows] = (rate * dwrite)[..., 0]
        out["dbeta"][rows] = (dwrite * miss).sum(dim=(-2, -1))
        out["dg"][rows] = (dfaded * faded).sum(dim=(-2, -1))
        d[:live] = dfaded * decay
    dinit = torch.empty_like(d)
    dinit[order] = d
    for name in ("dq", "dk"):
        out[name] = out[name].view(cu[-1], groups, wide, n).sum(dim=2)
    return {"dinit": dinit, **{name: t.view(s[name[1:]].shape) for name, t in out.items()}}
