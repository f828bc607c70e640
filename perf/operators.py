"""Cases and plain forms of the transformer-block operators.

Three operators and their gradients, as they stand between two FP8 linear layers:

  norm_fwd, norm_bwd  layer norm; its normalised rows may be kept as 8-bit codes with one
                      multiplier per 128 columns of a row, and the backward pass reads either
                      the input or those codes
  act_fwd, act_bwd    an activation f(a), or gated f(a) * b, whose inputs may be kept the same way
  moe_fwd, moe_bwd    token choices sorted by expert (each expert's segment padded to a multiple
                      of `align` rows), rows copied to their segments, expert outputs combined
                      with the router's weights; and the gradients of the last two

``own`` False: elementary torch operations in 32 bits, rounded once at the end.  ``own`` True:
the package's entry points.  ``exact`` is each operator's definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}
_FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FLT_MAX = torch.finfo(torch.float32).max
_EPS = 1e-5


def _norm(op, rows, cols, dtype="bf16", wdtype="fp32", ckpt="", pad=0, **k):
    """ckpt: the format of the 8-bit copy ("" for none); pad: columns by which the input's row stride exceeds cols."""
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, wdtype=wdtype, ckpt=ckpt, pad=pad, **k)


def _act(op, rows, cols, kind, gated, dtype="bf16", ckpt="", **k):
    return dict(op=op, rows=rows, cols=cols, kind=kind, gated=gated, dtype=dtype, ckpt=ckpt, **k)


def _moe(op, tokens, k, experts, hidden, align, dtype="bf16", ids="int64", **kw):
    return dict(op=op, tokens=tokens, k=k, experts=experts, hidden=hidden, align=align, dtype=dtype, ids=ids, **kw)


def listed():
    return [
        # one decoded token before a 4096-wide linear: latency only
        _norm("norm_fwd", 1, 4096, name="norm_fwd_token"),
        # the norm before a 4096-wide linear with 8192 tokens, its rows kept in 8 bits for training
        _norm("norm_fwd", 8192, 4096, ckpt="e4m3", name="norm_fwd_train"),
        # a ragged batch in binary32 with an odd width and a row stride of its own (a slice of a wider tensor)
        _norm("norm_fwd", 509, 1003, dtype="fp32", ckpt="e4m3", pad=6, name="norm_fwd_ragged"),
        # the backward pass of the 8192-token norm, from its 8-bit rows
        _norm("norm_bwd", 8192, 4096, ckpt="e4m3", name="norm_bwd_train"),
        # the widest norm of the GPT-sized linears, 2048 tokens, backward from the kept input
        _norm("norm_bwd", 2048, 12288, name="norm_bwd_wide"),
        # one decoded token through a gated SiLU between 11008-wide linears: latency only
        _act("act_fwd", 1, 11008, "silu", True, name="act_fwd_token"),
        # the same with 8192 tokens, both inputs kept in 8 bits for training
        _act("act_fwd", 8192, 11008, "silu", True, ckpt="e4m3", name="act_fwd_train"),
        # and its backward pass from the 8-bit inputs
        _act("act_bwd", 8192, 11008, "silu", True, ckpt="e4m3", name="act_bwd_train"),
        # a plain GELU between the 49152-wide linears of a GPT-sized layer, 2048 tokens, backward from the kept input
        _act("act_bwd", 2048, 49152, "gelu", False, name="act_bwd_gelu"),
        # one decoded token sent to 2 of 8 experts: three short launches
        _moe("moe_fwd", 1, 2, 8, 4096, 1, ids="int32", name="moe_fwd_token"),
        # 8192 tokens sent to 2 of 8 experts, segments padded to the FP8 GEMM's 128 rows
        _moe("moe_fwd", 8192, 2, 8, 4096, 128, name="moe_fwd_train"),
        # the gradients with many small experts: 8 of 64, an odd token count
        _moe("moe_bwd", 2047, 8, 64, 4096, 128, name="moe_bwd_fine"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "act_fwd", "act_bwd", "moe_fwd", "moe_bwd"))
    dtype = "bf16" if rng.random() < 0.7 else "fp32"
    ckpt = rng.choice(("", "e4m3", "e4m3", "e5m2"))
    if op.startswith("norm"):
        # any width two times in five, else a multiple of 128 as most models have
        cols = _log(rng, 64, 16384)
        cols = cols if rng.random() < 0.4 else max(64, cols // 128 * 128)
        rows = _log(rng, 1, min(32768, 50_000_000 // cols))
        return _norm(op, rows, cols, dtype, rng.choice(("bf16", "fp32")), ckpt, rng.choice((0, 0, 0, 8, 3)))
    if op.startswith("act"):
        gated = rng.random() < 0.7
        cols = _log(rng, 64, 49152)
        cols = cols if rng.random() < 0.4 else max(64, cols // 128 * 128)
        most = 40_000_000 if dtype == "fp32" else 80_000_000
        rows = _log(rng, 1, max(1, min(32768, most // cols)))
        return _act(op, rows, cols, rng.choice(("silu", "gelu", "gelu_tanh")), gated, dtype, ckpt)
    k = rng.choice((1, 2, 4, 6, 8))
    experts = max(k, _log(rng, 2, 256))
    hidden = _log(rng, 64, 8192)
    hidden = hidden if rng.random() < 0.4 else max(64, hidden // 64 * 64)
    align = rng.choice((1, 128))
    most = (70_000_000 if dtype == "bf16" else 35_000_000) // hidden - experts * align
    tokens = _log(rng, 1, max(1, min(16384, most // (2 * k + 2))))
    return _moe(op, tokens, k, experts, hidden, align, dtype, rng.choice(("int32", "int64")))


# ------------------------------------------------------------------ inputs
def _groups(cols):
    return (cols + 127) // 128


def _capacity(c):
    n = c["tokens"] * c["k"]
    return (n + min(n, c["experts"]) * (c["align"] - 1)) // c["align"] * c["align"]


def _codes(v, fmt):
    """8-bit values of v [rows, cols] float32 and the multiplier of every 128 columns of a row."""
    rows, cols = v.shape
    wide = torch.zeros(rows, _groups(cols) * 128, device=v.device)
    wide[:, :cols] = v
    wide = wide.view(rows, -1, 128)
    amax = wide.abs().amax(2)
    scale = torch.where((amax > 0) & (amax < math.inf), (_FMAX[fmt] / amax).clamp(max=_FLT_MAX), 1.0)
    codes = (wide * scale[..., None]).clamp(-_FMAX[fmt], _FMAX[fmt]).view(rows, -1)[:, :cols].to(_F8[fmt])
    return codes, 1.0 / scale


def _values(codes, mult):
    return codes.float() * mult.repeat_interleave(128, 1)[:, : codes.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = case
    dt = _DT[c["dtype"]]

    def normal(*shape, to=dt, sigma=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * sigma).to(to)

    s = dict(case=dict(c))
    if c["op"].startswith("norm"):
        rows, cols, wdt = c["rows"], c["cols"], _DT[c["wdtype"]]
        # a residual stream: 1 % of its columns are much larger, and rows have a mean of their own
        big = torch.rand(cols, generator=g, device="cuda") < 0.01
        wide = torch.randn((rows, cols + c["pad"]), generator=g, device="cuda")
        wide[:, :cols] *= torch.where(big, 20.0, 1.0)
        wide += 0.3 * torch.randn((rows, 1), generator=g, device="cuda")
        s["x"] = wide.to(dt)[:, :cols]
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(wdt)
        s["bias"] = normal(cols, to=wdt, sigma=0.1)
        if c["op"] == "norm_bwd":
            x = s["x"].float()
            mean = x.mean(1)
            rstd = 1 / (x - mean[:, None]).square().mean(1).add(_EPS).sqrt()
            s["dy"] = normal(rows, cols, sigma=1e-3)
            s["mean"], s["rstd"] = mean, rstd
            if c["ckpt"]:
                s["codes"], s["mult"] = _codes((x - mean[:, None]) * rstd[:, None], c["ckpt"])
                del s["x"], s["mean"]
    elif c["op"].startswith("act"):
        rows, cols = c["rows"], c["cols"]
        h = normal(rows, cols * (2 if c["gated"] else 1), sigma=1.5)
        a, b = h[:, :cols], h[:, cols:] if c["gated"] else None
        if c["op"] == "act_bwd":
            s["dy"] = normal(rows, cols, sigma=1e-3)
        if c["op"] == "act_bwd" and c["ckpt"]:
            s["a8"] = _codes(a.float(), c["ckpt"])
            s["b8"] = _codes(b.float(), c["ckpt"]) if c["gated"] else (None, None)
        else:
            s["a"], s["b"] = a, b
    else:
        t, k, e, h = c["tokens"], c["k"], c["experts"], c["hidden"]
        # a router that prefers some experts; about 3 % of the choices are dropped (id -1)
        logits = torch.randn((t, e), generator=g, device="cuda") + 0.7 * torch.randn(e, generator=g, device="cuda")
        top = logits.topk(k, 1)
        s["weights"] = torch.softmax(top.values, 1)
        drop = torch.rand((t, k), generator=g, device="cuda") < 0.03
        s["experts"] = torch.where(drop, -1, top.indices).to(torch.int32 if c["ids"] == "int32" else torch.int64)
        s["ys"] = normal(_capacity(c), h)
        if c["op"] == "moe_fwd":
            s["x"] = normal(t, h)
        else:
            s["dy"] = normal(t, h, sigma=1e-3)
            s["dxs"] = normal(_capacity(c), h, sigma=1e-3)
            s["offsets"], s["pos"], s["src"] = _route(s["experts"], e, c["align"], _capacity(c))
    return s


# ------------------------------------------------------------------ plain forms
def _norm_fwd(s):
    c, x = s["case"], s["x"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = 1 / ((d * d).mean(1, keepdim=True) + _EPS).sqrt()
    xh = d * rstd
    out = {"y": (xh * s["weight"].float() + s["bias"].float()).to(s["x"].dtype)}
    if c["ckpt"]:
        out["mean"], out["rstd"] = x.mean(1), rstd[:, 0]
        out["codes"], out["mult"] = _codes(xh, c["ckpt"])
    return out


def _norm_bwd(s):
    c, dy, rstd = s["case"], s["dy"].float(), s["rstd"][:, None]
    xh = _values(s["codes"], s["mult"]) if c["ckpt"] else (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    wdt = s["weight"].dtype
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xh).sum(0).to(wdt), "dbias": dy.sum(0).to(wdt)}


def _f(kind, x):
    """f(x) and f'(x)."""
    if kind == "gelu":
        cdf = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
        return x * cdf, cdf + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        two_k = 2 * math.sqrt(2 / math.pi)
        sg = 1 / (1 + torch.exp(-two_k * (x + 0.044715 * x * x * x)))
        return x * sg, sg + x * sg * (1 - sg) * two_k * (1 + 3 * 0.044715 * x * x)
    sg = 1 / (1 + torch.exp(-x))
    return x * sg, sg * (1 + x * (1 - sg))


def _act_fwd(s):
    c = s["case"]
    f, _ = _f(c["kind"], s["a"].float())
    out = {"y": (f * s["b"].float() if c["gated"] else f).to(s["a"].dtype)}
    if c["ckpt"]:
        out["a_codes"], out["a_mult"] = _codes(s["a"].float(), c["ckpt"])
        if c["gated"]:
            out["b_codes"], out["b_mult"] = _codes(s["b"].float(), c["ckpt"])
    return out


def _act_bwd(s):
    c, dy = s["case"], s["dy"].float()
    a = _values(*s["a8"]) if c["ckpt"] else s["a"].float()
    f, df = _f(c["kind"], a)
    if not c["gated"]:
        return {"da": (dy * df).to(s["dy"].dtype)}
    b = _values(*s["b8"]) if c["ckpt"] else s["b"].float()
    return {"da": (dy * b * df).to(s["dy"].dtype), "db": (dy * f).to(s["dy"].dtype)}


def _route(experts, n_experts, align, capacity):
    """Segment starts [E + 1], destination row of every choice (-1: dropped), source choice of every row (-1: padding)."""
    e = experts.reshape(-1)
    n, dev = e.numel(), e.device
    key = torch.where((e >= 0) & (e < n_experts), e, n_experts).to(torch.int64)
    key, order = torch.sort(key, stable=True)
    starts = torch.searchsorted(key, torch.arange(n_experts + 1, device=dev))
    padded = (starts.diff() + align - 1) // align * align
    offsets = torch.zeros(n_experts + 1, dtype=torch.int64, device=dev)
    offsets[1:] = padded.cumsum(0)
    row = offsets[key] + torch.arange(n, device=dev) - starts[key]
    kept = key < n_experts
    pos = torch.empty(n, dtype=torch.int64, device=dev)
    pos[order] = torch.where(kept, row, -1)
    src = torch.full((capacity + 1,), -1, dtype=torch.int64, device=dev)
    src[torch.where(kept, row, capacity)] = torch.where(kept, order, -1)
    return offsets.int(), pos.view(experts.shape).int(), src[:capacity].int()


def _gather(ys, pos, weights):
    """sum_j w[t, j] ys[pos[t, j]] over the choices that were not dropped, in 32 bits."""
    rows = ys[pos.clamp(min=0).long()].float()
    return torch.where(pos[..., None] >= 0, rows * weights[..., None] if weights is not None else rows, 0.0).sum(1)


def _moe_fwd(s):
    c = s["case"]
    offsets, pos, src = _route(s["experts"], c["experts"], c["align"], _capacity(c))
    xs = torch.where(src[:, None] >= 0, s["x"][src.clamp(min=0).long() // c["k"]], 0)
    y = _gather(s["ys"], pos, s["weights"]).to(s["x"].dtype)
    return {"offsets": offsets, "pos": pos, "src": src, "xs": xs, "y": y}


def _moe_bwd(s):
    c, pos, src, dy = s["case"], s["pos"], s["src"].long(), s["dy"].float()
    at = src.clamp(min=0)
    dys = torch.where(src[:, None] >= 0, dy[at // c["k"]] * s["weights"].reshape(-1)[at][:, None], 0.0)
    dots = (s["ys"][pos.clamp(min=0).long()].float() * dy[:, None]).sum(2)
    return {"dys": dys.to(s["dy"].dtype), "dweights": torch.where(pos >= 0, dots, 0.0),
            "dx": _gather(s["dxs"], pos, None).to(s["dy"].dtype)}


# ------------------------------------------------------------------ the package's operators
def _fmt(fq, name):
    return {"": None, "e4m3": fq.Format.E4M3, "e5m2": fq.Format.E5M2}[name]


def _own(s):
    import scaled_quantize_gemm_amax_gb300 as fq

    c = s["case"]
    if c["op"] == "norm_fwd":
        fmt = _fmt(fq, c["ckpt"])
        y, mean, rstd, q, mult = fq.layer_norm(s["x"], s["weight"], s["bias"], _EPS, checkpoint=fmt,
                                               stats=fmt is not None)
        return {"y": y, "mean": mean, "rstd": rstd, "codes": q.view(_F8[c["ckpt"]]), "mult": mult} if c["ckpt"] else {"y": y}
    if c["op"] == "norm_bwd":
        if c["ckpt"]:
            dx, dw, db = fq.layer_norm_backward(s["dy"], s["rstd"], s["weight"], q=s["codes"], s=s["mult"],
                                                fmt=_fmt(fq, c["ckpt"]))
        else:
            dx, dw, db = fq.layer_norm_backward(s["dy"], s["rstd"], s["weight"], x=s["x"], mean=s["mean"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if c["op"].startswith("act"):
        kind = {"silu": fq.Activation.SILU, "gelu": fq.Activation.GELU, "gelu_tanh": fq.Activation.GELU_TANH}[c["kind"]]
    if c["op"] == "act_fwd":
        y, qa, sa, qb, sb = fq.gated_act(s["a"], s["b"], kind, checkpoint=_fmt(fq, c["ckpt"]))
        out = {"y": y}
        if c["ckpt"]:
            out.update(a_codes=qa.view(_F8[c["ckpt"]]), a_mult=sa)
            if c["gated"]:
                out.update(b_codes=qb.view(_F8[c["ckpt"]]), b_mult=sb)
        return out
    if c["op"] == "act_bwd":
        if c["ckpt"]:
            da, db = fq.gated_act_backward(s["dy"], kind, qa=s["a8"][0], sa=s["a8"][1], qb=s["b8"][0], sb=s["b8"][1],
                                           fmt=_fmt(fq, c["ckpt"]))
        else:
            da, db = fq.gated_act_backward(s["dy"], kind, a=s["a"], b=s["b"])
        return {"da": da, "db": db} if c["gated"] else {"da": da}
    if c["op"] == "moe_fwd":
        route = fq.moe_route(s["experts"], c["experts"], c["align"])
        xs = fq.moe_dispatch(s["x"], route)
        y = fq.moe_combine(s["ys"], route, s["weights"])
        return {"offsets": route.offsets, "pos": route.pos, "src": route.src, "xs": xs, "y": y}
    route = fq.MoeRoute(s["offsets"], s["pos"], s["src"])
    dys, dw = fq.moe_combine_backward(s["dy"], s["ys"], route, s["weights"])
    return {"dys": dys, "dweights": dw, "dx": fq.moe_dispatch_backward(s["dxs"], route)}


_PLAIN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "act_fwd": _act_fwd, "act_bwd": _act_bwd,
          "moe_fwd": _moe_fwd, "moe_bwd": _moe_bwd}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = _SIZE[c["dtype"]]
    if c["op"].startswith(("norm", "act")):
        n = c["rows"] * c["cols"]
        kept = n + 4 * c["rows"] * _groups(c["cols"])   # one 8-bit copy
    if c["op"] == "norm_fwd":
        params = 2 * c["cols"] * _SIZE[c["wdtype"]]
        return {"bytes": 2 * n * e + params + (kept + 8 * c["rows"] if c["ckpt"] else 0), "flops": 8 * n}
    if c["op"] == "norm_bwd":
        params = 3 * c["cols"] * _SIZE[c["wdtype"]]
        return {"bytes": 2 * n * e + params + (kept + 4 * c["rows"] if c["ckpt"] else n * e + 8 * c["rows"]), "flops": 13 * n}
    sides = 2 if c.get("gated") else 1
    if c["op"] == "act_fwd":
        return {"bytes": (sides + 1) * n * e + (sides * kept if c["ckpt"] else 0), "flops": 8 * n}
    if c["op"] == "act_bwd":
        return {"bytes": (1 + sides) * n * e + sides * (kept if c["ckpt"] else n * e), "flops": 14 * n}
    rows, cap = c["tokens"] * c["k"], _capacity(c)
    one = c["hidden"] * e
    if c["op"] == "moe_fwd":
        ints = rows * (4 if c["ids"] == "int32" else 8) + 4 * (rows + cap + c["experts"] + 1)
        return {"bytes": (2 * c["tokens"] + cap + rows) * one + ints + 4 * rows, "flops": 2 * rows * c["hidden"]}
    return {"bytes": (2 * c["tokens"] + 2 * rows + cap) * one + 4 * (3 * rows + cap), "flops": 4 * rows * c["hidden"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_multipliers(v, fmt):
    rows, cols = v.shape
    amax = torch.stack([p.abs().amax(1) for p in v.split(128, 1)], 1)
    return torch.where(amax > 0, 1 / (_FMAX[fmt] / amax), 1.0)


def _exact_values(pair):
    codes, mult = pair
    return torch.cat([p.double() * mult[:, i:i + 1].double() for i, p in enumerate(codes.float().split(128, 1))], 1)


def _exact_act(kind, a):
    if kind == "silu":
        return torch.nn.functional.silu(a)
    return torch.nn.functional.gelu(a, approximate="tanh" if kind == "gelu_tanh" else "none")


def exact(case, seed):
    """The operators in 64 bits, by the library's own functions and differentiation where it has them.  The 8-bit codes
    themselves have no entry: which of two codes a value between them takes is a matter of the working precision."""
    c, s = case, prepare(case, seed)
    if c["op"] == "norm_fwd":
        x = s["x"].double()
        y = torch.nn.functional.layer_norm(x, (c["cols"],), s["weight"].double(), s["bias"].double(), _EPS)
        if not c["ckpt"]:
            return {"y": y}
        std = (x.var(1, unbiased=False) + _EPS).sqrt()
        xh = (x - x.mean(1, keepdim=True)) / std[:, None]
        return {"y": y, "mean": x.mean(1), "rstd": 1 / std, "codes": None, "mult": _exact_multipliers(xh, c["ckpt"])}
    if c["op"] == "norm_bwd":
        dy, w, rstd = s["dy"].double(), s["weight"].double(), s["rstd"].double()
        if c["ckpt"]:
            xh = _exact_values((s["codes"], s["mult"]))
        else:
            xh = (s["x"].double() - s["mean"].double()[:, None]) * rstd[:, None]
        n = c["cols"]
        dx = dy * w - (dy @ w / n)[:, None] - xh * (((dy * xh) @ w) / n)[:, None]
        return {"dx": dx * rstd[:, None], "dweight": torch.einsum("tc,tc->c", dy, xh), "dbias": dy.sum(0)}
    if c["op"] == "act_fwd":
        a = s["a"].double()
        y = _exact_act(c["kind"], a)
        out = {"y": y * s["b"].double() if c["gated"] else y}
        if c["ckpt"]:
            out.update(a_codes=None, a_mult=_exact_multipliers(a, c["ckpt"]))
            if c["gated"]:
                out.update(b_codes=None, b_mult=_exact_multipliers(s["b"].double(), c["ckpt"]))
        return out
    if c["op"] == "act_bwd":
        a = (_exact_values(s["a8"]) if c["ckpt"] else s["a"].double()).requires_grad_(True)
        dy = s["dy"].double()
        y = _exact_act(c["kind"], a)
        if not c["gated"]:
            return {"da": torch.autograd.grad(y, a, dy)[0]}
        b = _exact_values(s["b8"]) if c["ckpt"] else s["b"].double()
        return {"da": torch.autograd.grad(y, a, dy * b)[0], "db": dy * y.detach()}
    t, k, n_experts, align, cap = c["tokens"], c["k"], c["experts"], c["align"], _capacity(c)
    # the routing by one list per expert, on the host
    ids = s["experts"].reshape(-1).tolist()
    lists = [[] for _ in range(n_experts)]
    for i, e in enumerate(ids):
        if 0 <= e < n_experts:
            lists[e].append(i)
    offsets, pos, src = [0], [-1] * (t * k), [-1] * cap
    for one in lists:
        for rank, i in enumerate(one):
            pos[i] = offsets[-1] + rank
            src[pos[i]] = i
        offsets.append(offsets[-1] + -(-len(one) // align) * align)
    # each choice as an entry of a sparse matrix over the segment rows
    made = torch.tensor([i for i in range(t * k) if pos[i] >= 0], dtype=torch.int64, device="cuda")
    row = torch.tensor(pos, device="cuda")[made]
    w = s["weights"].double().reshape(-1)
    if c["op"] == "moe_fwd":
        xs = torch.zeros(cap, c["hidden"], dtype=torch.float64, device="cuda")
        xs[row] = s["x"].double()[made // k]
        y = torch.zeros(t, c["hidden"], dtype=torch.float64, device="cuda")
        y.index_add_(0, made // k, s["ys"].double()[row] * w[made, None])
        ints = {"offsets": offsets, "pos": pos, "src": src}
        ints = {n: torch.tensor(v, dtype=torch.int32) for n, v in ints.items()}
        return {**ints, "pos": ints["pos"].view(t, k), "xs": xs, "y": y}
    dy = s["dy"].double()
    dys = torch.zeros(cap, c["hidden"], dtype=torch.float64, device="cuda")
    dys[row] = dy[made // k] * w[made, None]
    dw = torch.zeros(t * k, dtype=torch.float64, device="cuda")
    dw[made] = torch.einsum("ih,ih->i", s["ys"].double()[row], dy[made // k])
    dx = torch.zeros(t, c["hidden"], dtype=torch.float64, device="cuda")
    dx.index_add_(0, made // k, s["dxs"].double()[row])
    return {"dys": dys, "dweights": dw.view(t, k), "dx": dx}
