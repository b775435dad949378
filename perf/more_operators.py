"""Cases of the operators of a training block around the expert layer: the root-mean-square norm with the residual's
addition and an MXFP8 output, activations kept in MXFP8 between the forward and the backward, and the softmax cross
entropy over a vocabulary, each with its backward.

``own`` chooses what ``run`` computes with: False, the plain form in elementary torch operations (fp32, fp64 where
fp32 loses what matters); True, the framework's own calls."""

import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6


# --- the cases -----------------------------------------------------------------
def listed():
    return [
        # the norm
        # one token of a decoding sequence, the SwiGLU layer workload's hidden size; launch latency is all of it
        {"name": "norm_token", "kind": "norm", "rows": 1, "cols": 7168, "stream": "bf16", "residual": True, "y": True,
         "mx": True},
        # the SwiGLU layer workload's tokens: the bf16 rows go to the gate, the codes to the permute
        {"name": "norm_train", "kind": "norm", "rows": 32768, "cols": 7168, "stream": "bf16", "residual": True,
         "y": True, "mx": True},
        # its backward: a ragged number of rows of the mid workload's size, the stream held in fp32
        {"name": "norm_bwd_odd", "kind": "norm_bwd", "rows": 1001, "cols": 2048, "stream": "f32", "dsum": True},
        # the training batch, the gradient of the residual stream added
        {"name": "norm_bwd_train", "kind": "norm_bwd", "rows": 32768, "cols": 7168, "stream": "bf16", "dsum": True},
        # activations kept in 8 bits
        # the forward's part: a few tokens, the mid workload's ffn; a quarter of the SwiGLU layer workload's tokens
        {"name": "keep_small", "kind": "keep", "T": 100, "k": 2, "E": 8, "F": 1408},
        {"name": "keep_train", "kind": "keep", "T": 8192, "k": 8, "E": 64, "F": 2048},
        # the backward's part: from what was kept to the operands of the products and the router's gradient
        {"name": "kept_bwd_small", "kind": "kept_bwd", "T": 100, "k": 2, "E": 8, "F": 1408, "H": 2048},
        {"name": "kept_bwd_train", "kind": "kept_bwd", "T": 8192, "k": 8, "E": 64, "F": 2048, "H": 7168},
        # the loss
        # the log probability of one token, the large workload's hidden size
        {"name": "xent_token", "kind": "xent", "rows": 1, "vocab": 65536, "k": 5120, "grad": False, "ignored": 0,
         "weighted": False},
        # scoring of a text with an odd vocabulary, a few positions masked
        {"name": "xent_score", "kind": "xent", "rows": 1000, "vocab": 32003, "k": 2048, "grad": False, "ignored": 37,
         "weighted": False},
        # a small training batch, odd everywhere, rows weighted and masked
        {"name": "xent_grad_odd", "kind": "xent", "rows": 257, "vocab": 10007, "k": 1024, "grad": True, "ignored": 30,
         "weighted": True},
        # a training batch
        {"name": "xent_train", "kind": "xent", "rows": 4096, "vocab": 65536, "k": 5120, "grad": True, "ignored": 0,
         "weighted": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("norm", "norm_bwd", "keep", "kept_bwd", "xent", "xent"))
    while True:
        if kind in ("norm", "norm_bwd"):
            c = {"kind": kind, "rows": _log(rng, 1, 32768), "cols": 32 * _log(rng, 4, 512),
                 "stream": rng.choice(("bf16", "bf16", "f32"))}
            if kind == "norm":
                c["residual"], c["mx"] = rng.random() < 0.7, rng.random() < 0.7
                c["y"] = not c["mx"] or rng.random() < 0.7
            else:
                c["dsum"] = rng.random() < 0.7
            # (the fp32 stream moves up to 1.6 times the bytes)
            if c["rows"] * c["cols"] * (1 if c["stream"] == "bf16" else 2) <= 32768 * 7168:
                return c
        elif kind in ("keep", "kept_bwd"):
            c = {"kind": kind, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "E": _log(rng, 1, 128),
                 "F": 32 * _log(rng, 1, 256)}
            c["k"] = min(c["k"], c["E"])
            if kind == "kept_bwd":
                c["H"] = 32 * _log(rng, 2, 256)
            if (c["T"] * c["k"] + 32 * c["E"]) * max(c["F"] / 2048, c.get("H", 0) / 7168) <= 8192 * 8 + 32 * 64:
                return c
        else:
            c = {"kind": kind, "rows": _log(rng, 1, 8192), "vocab": _log(rng, 500, 131072), "k": 32 * _log(rng, 2, 224),
                 "grad": rng.random() < 0.5, "ignored": 0, "weighted": rng.random() < 0.5}
            if rng.random() < 0.4:
                c["ignored"] = rng.randint(0, c["rows"])
            if rng.random() < 0.5:
                c["vocab"] = -(-c["vocab"] // 64) * 64
            if c["rows"] * c["vocab"] * c["k"] <= 4096 * 65536 * 5120 and c["rows"] * c["vocab"] <= 2 ** 29 \
                    and c["vocab"] * c["k"] <= 65536 * 5120:
                return c


def _cap(c):
    """Rows of the permuted buffers: every expert's rows padded to a multiple of 32."""
    return -(-(c["T"] * c["k"] + 31 * c["E"]) // 32) * 32


def work(case):
    c, mx = case, 33 / 32
    if c["kind"] in ("norm", "norm_bwd"):
        n, s = c["rows"] * c["cols"], 2 if c["stream"] == "bf16" else 4
        if c["kind"] == "norm":
            per = 2 + (2 * s if c["residual"] else 0) + (2 if c["y"] else 0) + (mx if c["mx"] else 0)
            return {"bytes": per * n + 4 * c["cols"], "flops": 8.0 * n}
        per = 2 + s * (3 if c["dsum"] else 2) + (2 if s == 4 else 0)
        return {"bytes": per * n + 8 * c["cols"], "flops": 16.0 * n}
    if c["kind"] == "keep":
        return {"bytes": _cap(c) * c["F"] * (4 + 3 * mx), "flops": 10.0 * _cap(c) * c["F"]}
    if c["kind"] == "kept_bwd":
        pairs = c["T"] * c["k"]
        glue = _cap(c) * c["F"] * (2 * mx + 2 + 5 * mx)
        return {"bytes": glue + c["T"] * c["H"] * mx + _cap(c) * (c["H"] * mx + 4) + 4 * pairs * 3 + 4 * c["T"] * c["E"],
                "flops": 20.0 * _cap(c) * c["F"] + 2.0 * _cap(c) * c["H"]}
    m, v, k = c["rows"], c["vocab"], c["k"]
    b = 2 * k * (m + v) + 4 * m * (3 + int(c["weighted"]))
    return {"bytes": b + (2 * k * (m + v) if c["grad"] else 0), "flops": (6.0 if c["grad"] else 2.0) * m * v * k}


# --- inputs --------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(dtype)


def _two(e):
    """Exactly 2^e in fp32, e whole in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _mx(x):
    """fp32 [R, 32 b] -> E4M3 codes [R, 32 b] and the scale bytes in panels [ceil(b / 4), R, 4] (nearest even)."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, -127).clamp(-127, 127)     # floor(log2 amax) - 8
    q = (b * _two(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[1] % 4))
    return q, s.unflatten(1, (-1, 4)).permute(1, 0, 2).contiguous()


def _value(q, s):
    """The fp32 values of codes [R, C] with panel scales."""
    sc = s.permute(1, 0, 2).flatten(1)[:, :q.shape[1] // 32]
    return (q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * _two(sc.int() - 127).unsqueeze(-1)).flatten(-2)


def _route(g, c):
    """Expert choices of random logits, and where their rows go: (ids, weights, dst_row, src_row)."""
    T, k, E = c["T"], c["k"], c["E"]
    val, ids = torch.sort(_normal(g, T, E), dim=1, descending=True)
    w = torch.softmax(val[:, :k], 1)
    flat = ids[:, :k].reshape(-1)
    order = torch.argsort(flat, stable=True)
    count = torch.bincount(flat, minlength=E)
    padded = (count + 31) // 32 * 32
    start = torch.cumsum(padded, 0) - padded - (torch.cumsum(count, 0) - count)
    dst = torch.empty_like(flat)
    dst[order] = torch.arange(T * k, device=DEV) + start[flat[order]]
    src = torch.full((_cap(c),), -1, dtype=torch.int64, device=DEV)
    src[dst] = torch.arange(T * k, device=DEV) // k
    return ids[:, :k].int().contiguous(), w.contiguous(), dst.int(), src.int()


def prepare(case, seed):
    c, g, bf = case, _gen(seed), torch.bfloat16
    if c["kind"] in ("norm", "norm_bwd"):
        R, C, st = c["rows"], c["cols"], bf if c["stream"] == "bf16" else torch.float32
        s = {"weight": 1 + _normal(g, C, std=0.1)}
        if c["kind"] == "norm":
            s["x"] = _normal(g, R, C, dtype=bf)
            s["residual"] = _normal(g, R, C, std=2.0, dtype=st) if c["residual"] else None
        else:
            s["sum"], s["dy"] = _normal(g, R, C, std=2.0, dtype=st), _normal(g, R, C, std=1e-3, dtype=bf)
            s["dsum"] = _normal(g, R, C, std=1e-3, dtype=st) if c["dsum"] else None
    elif c["kind"] in ("keep", "kept_bwd"):
        ids, w, dst, src = _route(g, c)
        live = (src >= 0).unsqueeze(1)
        h = _normal(g, _cap(c), 2 * c["F"], dtype=bf) * live
        s = {"h": h}
        if c["kind"] == "kept_bwd":
            s = {"ids": ids, "w": w, "dst": dst, "src": src, "da": _normal(g, _cap(c), c["F"], std=1e-2, dtype=bf) * live}
            s["keep_q"], s["keep_s"] = _mx(h.float())
            s["xq"], s["xs"] = _mx(_normal(g, c["T"], c["H"], dtype=bf).float())
    else:
        m, v, k = c["rows"], c["vocab"], c["k"]
        s = {"x": _normal(g, m, k, dtype=bf), "w": _normal(g, v, k, std=3 * k ** -0.5, dtype=bf),
             "t": torch.randint(0, v, (m,), generator=g, device=DEV, dtype=torch.int32)}
        s["t"][torch.randperm(m, generator=g, device=DEV)[:c["ignored"]]] = -100
        s["rw"] = torch.rand(m, generator=g, device=DEV) / m if c["weighted"] else None
    s["case"] = dict(case)
    return s


# --- one pass ------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "keep": _own_keep, "kept_bwd": _own_kept_bwd,
                "xent": _own_xent}[c["kind"]](s, c)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "keep": _keep, "kept_bwd": _kept_bwd, "xent": _xent}[c["kind"]](s, c)


def _pair(q, s):
    """Codes and scales as the values they stand for."""
    return {"q": q.view(torch.float8_e4m3fn), "s": s.view(torch.float8_e8m0fnu)}


# --- plain forms ---------------------------------------------------------------
def _norm(s, c):
    r, st = s["x"].float(), torch.bfloat16 if c["stream"] == "bf16" else torch.float32
    out = {}
    if c["residual"]:
        out["sum"] = (r + s["residual"].float()).to(st)
        r = out["sum"].float()
    y = (r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["weight"]).to(torch.bfloat16)
    if c["y"]:
        out["y"] = y
    if c["mx"]:
        out["row"] = _pair(*_mx(y.float()))
    return out


def _norm_bwd(s, c):
    r, dy = s["sum"].float(), s["dy"].float()
    inv = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    n, g = r * inv, dy * s["weight"]
    d = inv * (g - n * (g * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        d = d + s["dsum"].float()
    out = {"dres": d.to(s["sum"].dtype), "dweight": (dy * n).sum(0, dtype=torch.float64).float()}
    if c["stream"] == "f32":                           # the branch in front takes its gradient in bf16
        out["dx"] = d.to(torch.bfloat16)
    return out


def _keep(s, c):
    h = s["h"].float()
    g, u = h[:, :c["F"]], h[:, c["F"]:]
    a = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
    return {"row": _pair(*_mx(a.float())), "keep": _pair(*_mx(h))}


def _kept_bwd(s, c):
    h, d = _value(s["keep_q"], s["keep_s"]), s["da"].float()
    g, u = h[:, :c["F"]], h[:, c["F"]:]
    sig = 1 / (1 + torch.exp(-g))
    a = g * sig * u
    dh = torch.cat([d * u * sig * (1 + g * (1 - sig)), d * g * sig], 1).to(torch.bfloat16).float()
    dots = (d * a).sum(1)[s["dst"].long()].view(c["T"], c["k"])
    dl = dots - s["w"] * dots.sum(1, keepdim=True)
    x = torch.where((s["src"] >= 0).unsqueeze(1), _value(s["xq"], s["xs"])[s["src"].clamp_min(0).long()], 0.0)
    return {"row": _pair(*_mx(dh)), "col": _pair(*_mx(dh.t().contiguous())),
            "a": _pair(*_mx(a.to(torch.bfloat16).float().t().contiguous())), "x": _pair(*_mx(x.t().contiguous())),
            "dlogits": torch.zeros(c["T"], c["E"], device=DEV).scatter_(1, s["ids"].long(), dl)}


def _xent(s, c):
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    t = s["t"].long().clamp_min(0).unsqueeze(1)
    live = (s["t"] >= 0).unsqueeze(1)
    out = {"loss": torch.where(live, lse - z.gather(1, t), 0.0).squeeze(1), "lse": lse.squeeze(1)}
    if c["grad"]:
        g = live.float() if s["rw"] is None else live * s["rw"].unsqueeze(1)
        dz = torch.exp(z - lse)
        dz = dz.scatter_add_(1, t, torch.full_like(lse, -1.0)).mul_(g)
        out["dx"], out["dw"] = (dz @ w).to(torch.bfloat16), (dz.t() @ x).to(torch.bfloat16)
    return out


# --- the framework's calls -----------------------------------------------------
def _lib():
    import mxfp8_block_scaled_07_amd as mxa
    return mxa


def _bytes(*shape):
    return torch.empty(*shape, dtype=torch.uint8, device=DEV)


def _mx_buffers(mxa, rows, cols):
    return _bytes(rows, cols), _bytes(*mxa.scale_shape(rows, cols))


def _own_norm(s, c):
    mxa = _lib()
    R, C = c["rows"], c["cols"]
    if "own" not in s:
        st = torch.bfloat16 if c["stream"] == "bf16" else torch.float32
        s["own"] = {"sum": torch.empty(R, C, dtype=st, device=DEV) if c["residual"] else None,
                    "y": torch.empty(R, C, dtype=torch.bfloat16, device=DEV) if c["y"] else None,
                    "row": _mx_buffers(mxa, R, C) if c["mx"] else (None, None)}
    o = s["own"]
    mxa.mx_rmsnorm(s["x"], s["residual"], mxa.MX_OUT_BF16 if c["stream"] == "bf16" else mxa.MX_OUT_F32, s["weight"], R,
                   C, EPS, o["sum"], o["y"], *o["row"])
    out = {k: o[k] for k in ("sum", "y") if o[k] is not None}
    if c["mx"]:
        out["row"] = _pair(*o["row"])
    return out


def _own_norm_bwd(s, c):
    mxa = _lib()
    R, C = c["rows"], c["cols"]
    if "own" not in s:
        wsb = mxa.mx_rmsnorm_bwd_workspace_size(R, C)
        s["own"] = {"dres": torch.empty_like(s["sum"]), "dweight": torch.empty(C, device=DEV), "wsb": wsb,
                    "ws": _bytes(max(wsb, 16)),
                    "dx": torch.empty(R, C, dtype=torch.bfloat16, device=DEV) if c["stream"] == "f32" else None}
    o = s["own"]
    mxa.mx_rmsnorm_bwd(s["dy"], s["sum"], s["dsum"], mxa.MX_OUT_BF16 if c["stream"] == "bf16" else mxa.MX_OUT_F32,
                       s["weight"], R, C, EPS, o["dres"], o["dx"], o["dweight"], o["ws"], o["wsb"])
    return {k: o[k] for k in ("dres", "dx", "dweight") if o[k] is not None}


def _own_keep(s, c):
    mxa = _lib()
    R, F = _cap(c), c["F"]
    if "own" not in s:
        s["own"] = {"row": _mx_buffers(mxa, R, F), "keep": _mx_buffers(mxa, R, 2 * F)}
    o = s["own"]
    mxa.mx_swiglu_keep(s["h"], R, F, *o["row"], *o["keep"])
    return {"row": _pair(*o["row"]), "keep": _pair(*o["keep"])}


def _own_kept_bwd(s, c):
    mxa = _lib()
    R, F, H, T, k, E = _cap(c), c["F"], c["H"], c["T"], c["k"], c["E"]
    if "own" not in s:
        wsb = mxa.mx_swiglu_bwd_kept_workspace_size(R, F)
        s["own"] = {"row": _mx_buffers(mxa, R, 2 * F), "col": _mx_buffers(mxa, 2 * F, R), "a": _mx_buffers(mxa, F, R),
                    "x": _mx_buffers(mxa, H, R), "dots": torch.empty(R, device=DEV), "wsb": wsb,
                    "ws": _bytes(max(wsb, 16)), "dlogits": torch.empty(T, E, device=DEV)}
    o = s["own"]
    mxa.mx_swiglu_bwd_kept(s["keep_q"], s["keep_s"], s["da"], R, F, *o["row"], *o["col"], *o["a"], o["dots"], o["ws"],
                           o["wsb"])
    mxa.mx_router_bwd_dots(o["dots"], R, s["dst"], s["ids"], s["w"], T, E, k, o["dlogits"])
    mxa.mx_requantize(s["xq"], s["xs"], T, H, s["src"], R, *o["x"])
    return {"row": _pair(*o["row"]), "col": _pair(*o["col"]), "a": _pair(*o["a"]), "x": _pair(*o["x"]),
            "dlogits": o["dlogits"]}


def _own_xent(s, c):
    mxa = _lib()
    m, v, k = c["rows"], c["vocab"], c["k"]
    if "own" not in s:
        wsb = mxa.mx_bf16_xent_workspace_size(m, v, k, int(c["grad"]))
        s["own"] = {"loss": torch.empty(m, device=DEV), "lse": torch.empty(m, device=DEV), "wsb": wsb,
                    "ws": _bytes(max(wsb, 16)),
                    "dx": torch.empty(m, k, dtype=torch.bfloat16, device=DEV) if c["grad"] else None,
                    "dw": torch.empty(v, k, dtype=torch.bfloat16, device=DEV) if c["grad"] else None}
    o = s["own"]
    mxa.mx_bf16_xent(s["x"], s["w"], s["t"], s["rw"], m, v, k, o["loss"], o["lse"], o["dx"], o["dw"], o["ws"], o["wsb"])
    return {n: o[n] for n in ("loss", "lse", "dx", "dw") if o[n] is not None}


# --- what the operators define, in 64 bits ---------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "keep": _exact_keep, "kept_bwd": _exact_kept_bwd,
            "xent": _exact_xent}[case["kind"]](s, case)


F64 = torch.float64


def _two64(e):
    """Exactly 2^e in fp64."""
    return ((e.long() + 1023) << 52).view(F64)


def _exact_mx(v):
    """fp64 [R, C] in units of its blocks' scales, as the codes stand for it before their rounding (a scale, a power of
    two that jumps where a largest value does, is compared between the sides alone)."""
    R, C = v.shape
    blocks = v.reshape(R, C // 32, 32)
    top = blocks.abs().amax(2)
    scale = _two64(torch.where(top > 0, torch.frexp(top).exponent - 9, -127).clamp(-127, 127))
    return {"q": (blocks / scale.unsqueeze(2)).clamp(-448, 448).reshape(R, C), "s": None}


def _exact_value(q, s):
    b = torch.arange(q.shape[1] // 32, device=DEV)
    scale = _two64(s[b // 4, :, b % 4].t().int() - 127)
    return q.view(torch.float8_e4m3fn).to(F64) * torch.repeat_interleave(scale, 32, dim=1)


def _bf16(v):
    """fp64 rounded to bf16 once (to nearest, halves to even)."""
    step = _two64(torch.frexp(v).exponent.clamp_min(-125) - 8)
    return torch.round(v / step) * step


def _exact_norm(s, c):
    r, out = s["x"].to(F64), {}
    if c["residual"]:
        r = r + s["residual"].to(F64)
        out["sum"] = r
        r = _bf16(r) if c["stream"] == "bf16" else r.float().to(F64)
    y = r / torch.sqrt(r.square().mean(1, keepdim=True) + EPS) * s["weight"].to(F64)
    if c["y"]:
        out["y"] = y
    if c["mx"]:
        out["row"] = _exact_mx(_bf16(y))
    return out


def _exact_norm_bwd(s, c):
    r = s["sum"].to(F64).requires_grad_()
    w = s["weight"].to(F64).requires_grad_()
    y = r / torch.sqrt(r.square().mean(1, keepdim=True) + EPS) * w
    d, dw = torch.autograd.grad(y, (r, w), s["dy"].to(F64))
    if c["dsum"]:
        d = d + s["dsum"].to(F64)
    return {"dres": d, "dweight": dw, "dx": d} if c["stream"] == "f32" else {"dres": d, "dweight": dw}


def _exact_keep(s, c):
    h = s["h"].to(F64)
    a = torch.nn.functional.silu(h[:, :c["F"]]) * h[:, c["F"]:]
    return {"row": _exact_mx(_bf16(a)), "keep": _exact_mx(h)}


def _exact_kept_bwd(s, c):
    h = _exact_value(s["keep_q"], s["keep_s"]).requires_grad_()
    a = torch.nn.functional.silu(h[:, :c["F"]]) * h[:, c["F"]:]
    d = s["da"].to(F64)
    dh = torch.autograd.grad(a, h, d)[0]
    a = a.detach()
    p = (a * d).sum(1)[s["dst"].long()].reshape(c["T"], c["k"])
    dl = torch.zeros(c["T"], c["E"], dtype=F64, device=DEV)
    dl[torch.arange(c["T"], device=DEV).unsqueeze(1), s["ids"].long()] = p - s["w"].to(F64) * p.sum(1, keepdim=True)
    x = torch.zeros(_cap(c), c["H"], dtype=F64, device=DEV)
    rows = torch.nonzero(s["src"] >= 0).squeeze(1)
    x[rows] = _exact_value(s["xq"], s["xs"])[s["src"][rows].long()]
    dh = _bf16(dh)
    return {"row": _exact_mx(dh), "col": _exact_mx(dh.t()), "a": _exact_mx(_bf16(a).t()), "x": _exact_mx(x.t()),
            "dlogits": dl}


def _exact_xent(s, c):
    x, w = s["x"].to(F64), s["w"].to(F64)
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    rows = torch.nonzero(s["t"] >= 0).squeeze(1)
    t = s["t"][rows].long()
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, t]
    if not c["grad"]:
        return {"loss": loss, "lse": lse}
    g = torch.zeros_like(lse)
    g[rows] = 1.0 if s["rw"] is None else s["rw"][rows].to(F64)
    z = torch.softmax(z, 1)
    z[rows, t] -= 1
    z *= g.unsqueeze(1)
    return {"loss": loss, "lse": lse, "dx": z @ w, "dw": z.t() @ x}
