"""Cases and plain forms of the operators of a mixture-of-experts training or serving step.

Three operators and their gradients, next to the FP8 linear layers and the expert routing:

  rms_fwd, rms_bwd       h = x + residual, y = h / sqrt(mean h^2 + eps) * weight; y leaves in the
                         data's type, in 8 bits with scales (what an FP8 product reads), or both
  group_fwd, group_dgrad, group_wgrad
                         products of FP8 matrices grouped by expert: rows sorted by expert, each
                         expert's segment a multiple of 128 rows, times that expert's weight; the
                         gradient of the rows; the gradient of every expert's weight
  clip                   the 2-norm over all of a model's gradients, and the gradients scaled so
                         that it is at most max_norm

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
_E8 = torch.float8_e8m0fnu
_FLT_MAX = torch.finfo(torch.float32).max
_EPS = 1e-5


def _rms(op, rows, cols, dtype="bf16", wdtype="fp32", residual=True, recipe="", fmt="e4m3", keep_y=True, pad=0, **k):
    """recipe: of y's 8-bit copy ("" for none); keep_y: y in the data's type too; pad: columns by which x's row stride exceeds cols."""
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, wdtype=wdtype, residual=residual, recipe=recipe, fmt=fmt,
                keep_y=keep_y or not recipe, pad=pad, **k)


def _group(op, tokens, k, experts, n, depth, recipe="mx", fa="e4m3", fb="e4m3", out="bf16", **kw):
    """group_fwd, group_dgrad: [rows, depth] times an expert's [n, depth]; group_wgrad: an expert's [n, rows] times [depth, rows]."""
    return dict(op=op, tokens=tokens, k=k, experts=experts, n=n, depth=depth, recipe=recipe, fa=fa, fb=fb, out=out, **kw)


def _clip(sizes, dtype="bf16", max_norm=1.0, **k):
    """sizes: the tensors' element counts, a text; dtype: bf16, fp32 or mixed (every third tensor fp32)."""
    return dict(op="clip", sizes=" ".join(str(s) for s in sizes), dtype=dtype, max_norm=max_norm, **k)


def listed():
    block = [4096 * 4096] * 4 + [4096 * 11008] * 3 + [4096] * 2   # a block of 4096-wide linears with an 11008-wide MLP
    return [
        # one decoded token before a 4096-wide linear, which reads its 8-bit row: latency only
        _rms("rms_fwd", 1, 4096, recipe="1x128", keep_y=False, name="rms_fwd_token"),
        # 8192 tokens before a 4096-wide MXFP8 linear: the residual stream in and out, 8-bit rows with tiled scales
        _rms("rms_fwd", 8192, 4096, recipe="mx_tiled", keep_y=False, name="rms_fwd_train"),
        # a ragged batch in binary32, odd width, a slice of a wider tensor, per-tensor scaling with the amax recorded
        _rms("rms_fwd", 509, 1003, dtype="fp32", recipe="tensor", pad=6, name="rms_fwd_ragged"),
        # the backward pass of the 8192-token norm, the residual stream's own gradient added
        _rms("rms_bwd", 8192, 4096, name="rms_bwd_train"),
        # the widest norm of the GPT-sized linears, 2048 tokens, no residual
        _rms("rms_bwd", 2048, 12288, residual=False, name="rms_bwd_wide"),
        # one decoded token at 2 of 8 experts' 4096 -> 11008 linears: two weights streamed
        _group("group_fwd", 1, 2, 8, 11008, 4096, name="group_fwd_token"),
        # 8192 tokens at 2 of 8 experts' 4096 -> 11008 linears
        _group("group_fwd", 8192, 2, 8, 11008, 4096, name="group_fwd_train"),
        # gradient of the rows with many small experts: 8 of 64, an odd token count, per-tensor scales, E5M2 gradients
        _group("group_dgrad", 2047, 8, 64, 4096, 2048, recipe="tensor", fa="e5m2", name="group_dgrad_fine"),
        # every expert's weight gradient of the 8192-token linears, binary32 out
        _group("group_wgrad", 8192, 2, 8, 11008, 4096, out="fp32", name="group_wgrad_train"),
        # a block's norms and router only: latency
        _clip([4096] * 4 + [8 * 4096] + [11008] * 2, max_norm=0.25, name="clip_small"),
        # four such blocks in one step
        _clip(block * 4, name="clip_model"),
        # many odd tensors, bf16 and binary32 mixed, views into flat buffers at any alignment
        _clip([1003 + 7919 * i % 65537 * 3 for i in range(300)], dtype="mixed", name="clip_ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rms_fwd", "rms_fwd", "rms_bwd", "group_fwd", "group_dgrad", "group_wgrad", "clip"))
    if op.startswith("rms"):
        dtype = "bf16" if rng.random() < 0.7 else "fp32"
        recipe = rng.choice(("", "tensor", "1x128", "mx", "mx_tiled"))
        cols = _log(rng, 64, 16384)
        if recipe == "mx_tiled":
            cols = max(128, cols // 128 * 128)
        elif recipe == "mx":
            cols = cols // 32 * 32
        elif rng.random() < 0.6:
            cols = max(64, cols // 128 * 128)
        rows = _log(rng, 1, min(32768, 33_000_000 // cols))
        rows = max(128, rows // 128 * 128) if recipe == "mx_tiled" else rows
        return _rms(op, rows, cols, dtype, rng.choice(("bf16", "fp32")), rng.random() < 0.7, recipe,
                    rng.choice(("e4m3", "e4m3", "e5m2")), rng.random() < 0.4, rng.choice((0, 0, 0, 8, 3)))
    if op == "clip":
        n = _log(rng, 1, 600)
        most = 600_000_000 // n
        sizes = [_log(rng, 1, most) for _ in range(n)]
        return _clip(sizes, rng.choice(("bf16", "bf16", "fp32", "mixed")), rng.choice((0.25, 1.0, 1e6)))
    experts = _log(rng, 1, 128)
    k = min(experts, rng.choice((1, 2, 4, 8)))
    depth = _log(rng, 1, 64) * 128
    n = _log(rng, 1, max(1, min(96, 2_800_000_000 // (experts * depth * 128)))) * 128
    most = 700_000_000_000 // (n * depth * k)
    tokens = _log(rng, 1, max(1, min(16384, most, 1_000_000_000 // (k * max(n, depth)))))
    grad = op != "group_fwd"
    return _group(op, tokens, k, experts, n, depth, rng.choice(("tensor", "mx")), rng.choice(("e4m3", "e5m2")) if grad else "e4m3",
                  "e4m3", rng.choice(("bf16", "fp32")))


# ------------------------------------------------------------------ inputs
def _mx_exponents(amax, fmt):
    """The smallest e with amax <= FMAX 2^e (FMAX = 1.75 2^top), 0 for 0."""
    m, e = torch.frexp(amax)
    e = e - 1 - (8 if fmt == "e4m3" else 15) + (m > 0.875).int()
    return torch.where((amax > 0) & (amax < math.inf), e.clamp(-127, 127), 0)


def _tiled(bytes_):
    """E8M0 bytes [rows, blocks] in the order that the products read: 512-byte atoms of 128 rows x 4 blocks."""
    r, b = bytes_.shape
    return bytes_.view(r // 128, 4, 32, b // 4, 4).permute(0, 3, 2, 1, 4).reshape(r // 128, b // 4, 512)


def _untiled(atoms):
    r, b = atoms.shape[0] * 128, atoms.shape[1] * 4
    return atoms.view(r // 128, b // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r, b)


def _quantise(v, recipe, fmt, scale=None):
    """v float32 [rows, cols] as (codes in the 8-bit type, multipliers): one a tensor (`scale` given), one a 1x128 or 1x32 block."""
    rows, cols = v.shape
    top = _FMAX[fmt]
    if recipe == "tensor":
        return (v * scale).clamp(-top, top).to(_F8[fmt]), 1.0 / scale
    width = 128 if recipe == "1x128" else 32
    blocks = -(-cols // width)
    wide = torch.zeros(rows, blocks * width, device=v.device)
    wide[:, :cols] = v
    wide = wide.view(rows, blocks, width)
    amax = wide.abs().amax(2)
    if recipe == "1x128":
        by = torch.where((amax > 0) & (amax < math.inf), (top / amax).clamp(max=_FLT_MAX), 1.0)
        mult = 1.0 / by
    else:
        e = _mx_exponents(amax, fmt)
        by = torch.ldexp(torch.ones_like(amax), -e)
        mult = (e + 127).to(torch.uint8)
        mult = (_tiled(mult) if recipe == "mx_tiled" else mult).view(_E8)
    codes = (wide * by[..., None]).clamp(-top, top).view(rows, -1)[:, :cols].to(_F8[fmt])
    return codes, mult


def _capacity(c):
    n = c["tokens"] * c["k"]
    return (n + min(n, c["experts"]) * 127) // 128 * 128


def _stack(v, recipe, fmt):
    """v [rows, cols] as an operand of the grouped products: codes and their per-tensor or tiled 1x32 multipliers."""
    if recipe == "mx":
        return _quantise(v, "mx_tiled", fmt)
    scale = (_FMAX[fmt] / v.abs().amax().clamp(min=1e-30)).reshape(1)
    return _quantise(v, "tensor", fmt, scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = case

    def normal(*shape, to=torch.float32, sigma=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * sigma).to(to)

    s = dict(case=dict(c))
    if c["op"].startswith("rms"):
        rows, cols, dt, wdt = c["rows"], c["cols"], _DT[c["dtype"]], _DT[c["wdtype"]]
        # a residual stream, 1 % of whose columns are much larger, and a block's output to be added to it
        big = torch.rand(cols, generator=g, device="cuda") < 0.01
        wide = normal(rows, cols + c["pad"])
        wide[:, :cols] *= torch.where(big, 20.0, 1.0)
        s["x"] = wide.to(dt)[:, :cols]
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(wdt)
        s["residual"] = normal(rows, cols, to=dt, sigma=0.3) if c["residual"] else None
        if c["op"] == "rms_bwd":
            h = s.pop("x").float() + s.pop("residual").float() if c["residual"] else s.pop("x").float()
            s["h"] = h.to(dt)
            s["rstd"] = 1 / s["h"].float().square().mean(1).add(_EPS).sqrt()
            s["dy"] = normal(rows, cols, to=dt, sigma=1e-3)
            s["dh"] = normal(rows, cols, to=dt, sigma=1e-3) if c["residual"] else None
        elif c["recipe"] == "tensor":
            s["scale"] = torch.full((1,), _FMAX[c["fmt"]] / 24.0, device="cuda")   # of past steps' largest values
    elif c["op"].startswith("group"):
        t, k, e, n, depth = c["tokens"], c["k"], c["experts"], c["n"], c["depth"]
        # a router that prefers some experts
        logits = normal(t, e) + 0.7 * normal(e)
        counts = torch.bincount(logits.topk(k, 1).indices.reshape(-1), minlength=e)
        padded = (counts + 127) // 128 * 128
        offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = padded.cumsum(0)
        s["offsets"] = offsets.int()
        # rows that hold a token; the others pad the segments and are 0
        cap = _capacity(c)
        row = torch.arange(cap, device="cuda")
        of = torch.searchsorted(offsets[1:], row, right=True).clamp(max=e - 1)
        held = (row - offsets[of] < counts[of]) & (row < offsets[-1])
        big = torch.where(torch.rand(depth, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        if c["op"] == "group_wgrad":   # column copies: gradients [n, rows] and inputs [depth, rows]
            s["a"], s["sa"] = _stack(normal(n, cap, sigma=1e-3) * held, c["recipe"], c["fa"])
            s["b"], s["sb"] = _stack(normal(depth, cap) * held * big[:, None], c["recipe"], c["fb"])
        else:
            x = normal(cap, depth) * big if c["op"] == "group_fwd" else normal(cap, depth, sigma=1e-3)
            s["a"], s["sa"] = _stack(x * held[:, None], c["recipe"], c["fa"])
            # the weights stacked by rows, or, as the column copy has them for the rows' gradient, by columns
            shape = (e * n, depth) if c["op"] == "group_fwd" else (n, e * depth)
            s["b"], s["sb"] = _stack(normal(*shape, sigma=0.02), c["recipe"], c["fb"])
    else:
        sizes = [int(v) for v in c["sizes"].split()]
        f32 = [c["dtype"] == "fp32" or c["dtype"] == "mixed" and i % 3 == 2 for i in range(len(sizes))]
        # gradients and their clipped copies as views into flat buffers
        for name, kind in (("fp32", True), ("bf16", False)):
            total = sum(n for n, f in zip(sizes, f32) if f == kind)
            s[name] = normal(total, to=_DT[name], sigma=2e-3) if total else None
            s[name + "_out"] = torch.empty_like(s[name]) if total else None
        at, s["grads"], s["outs"] = {True: 0, False: 0}, [], []
        for n, f in zip(sizes, f32):
            name = "fp32" if f else "bf16"
            s["grads"].append(s[name][at[f]:at[f] + n])
            s["outs"].append(s[name + "_out"][at[f]:at[f] + n])
            at[f] += n
    return s


# ------------------------------------------------------------------ plain forms
def _rms_fwd(s):
    c, dt = s["case"], _DT[s["case"]["dtype"]]
    out = {}
    h = s["x"].float()
    if c["residual"]:
        out["h"] = (h + s["residual"].float()).to(dt)   # the stream as it is kept, of which the norm is taken
        h = out["h"].float()
    rstd = 1 / ((h * h).mean(1, keepdim=True) + _EPS).sqrt()
    y = h * rstd * s["weight"].float()
    out["rstd"] = rstd[:, 0]
    if c["keep_y"]:
        out["y"] = y.to(dt)
    if c["recipe"]:
        out["codes"], mult = _quantise(y, c["recipe"], c["fmt"], s.get("scale"))
        if c["recipe"] == "tensor":
            out["amax"] = y.abs().amax().reshape(1)
        else:
            out["mult"] = mult
    return out


def _rms_bwd(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    xh = h * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xh).sum(0).to(s["weight"].dtype)}


def _values(codes, mult):
    """The values that per-tensor or tiled 1x32 codes stand for."""
    v = codes.float()
    if mult.dtype == torch.float32:
        return v * mult
    e = _untiled(mult.view(torch.uint8)).int() - 127
    return (v.view(v.shape[0], -1, 32) * torch.ldexp(torch.ones(e.shape, device=v.device), e)[..., None]).view(v.shape)


def _parts(s):
    """Every expert's rows, and the operands of its product."""
    c = s["case"]
    starts = s["offsets"].tolist()
    a, n, depth = _values(s["a"], s["sa"]), c["n"], c["depth"]
    for e in range(c["experts"]):
        lo, hi = starts[e], starts[e + 1]
        rows = slice(lo, hi)
        if c["op"] == "group_wgrad":
            yield e, rows, a[:, rows], None
        elif lo < hi:   # only the weights of experts with rows are widened
            tiled = s["sb"].dtype != torch.float32
            if c["op"] == "group_fwd":
                sb = s["sb"][e * n // 128:(e + 1) * n // 128] if tiled else s["sb"]
                b = _values(s["b"][e * n:(e + 1) * n], sb)
            else:
                sb = s["sb"][:, e * depth // 128:(e + 1) * depth // 128] if tiled else s["sb"]
                b = _values(s["b"][:, e * depth:(e + 1) * depth].contiguous(), sb.contiguous())
            yield e, rows, a[rows], b


def _product(s):
    c = s["case"]
    dt = _DT[c["out"]]
    if c["op"] == "group_wgrad":
        b = _values(s["b"], s["sb"])
        out = torch.empty(c["experts"], c["n"], c["depth"], dtype=dt, device="cuda")
        for e, rows, a, _ in _parts(s):
            out[e] = a @ b[:, rows].t()
        return {"dw": out}
    out = torch.zeros(s["a"].shape[0], c["n"], dtype=dt, device="cuda")   # rows behind the last segment: 0
    for _, rows, a, b in _parts(s):
        out[rows] = a @ b.t()
    return {"y": out}


def _clip_norm(s):
    c = s["case"]
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()
    coef = (c["max_norm"] / (total + 1e-6)).clamp(max=1.0)
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * coef)
    return _clipped(s, total.reshape(1))


def _clipped(s, norm):
    return {"norm": norm, **{n: s[n + "_out"] for n in ("bf16", "fp32") if s[n] is not None}}


# ------------------------------------------------------------------ the package's operators
def _own(s):
    import scaled_quantize_gemm_amax_gb300 as fq

    c = s["case"]
    fmt = {"e4m3": fq.Format.E4M3, "e5m2": fq.Format.E5M2}
    if c["op"] == "rms_fwd":
        recipe = {"": None, "tensor": fq.Recipe.TENSOR, "1x128": fq.Recipe.BLOCK_1x128, "mx": fq.Recipe.MX_1x32,
                  "mx_tiled": fq.Recipe.MX_1x32_TILED}[c["recipe"]]
        amax = torch.empty(1, device="cuda") if c["recipe"] == "tensor" else None
        y, h, rstd, q, m = fq.rms_norm(s["x"], s["weight"], s["residual"], _EPS, recipe=recipe, fmt=fmt[c["fmt"]],
                                       scale=s.get("scale"), amax_out=amax, keep_y=c["keep_y"])
        out = {"rstd": rstd}
        if c["residual"]:
            out["h"] = h
        if c["keep_y"]:
            out["y"] = y
        if c["recipe"]:
            out["codes"] = q.view(_F8[c["fmt"]])
            if c["recipe"] == "tensor":
                out["amax"] = amax
            else:
                out["mult"] = m if c["recipe"] == "1x128" else m.view(_E8)
        return out
    if c["op"] == "rms_bwd":
        dx, dw = fq.rms_norm_backward(s["dy"], s["h"], s["rstd"], s["weight"], dh=s["dh"])
        return {"dx": dx, "dweight": dw}
    if c["op"] == "clip":
        return _clipped(s, fq.clip_grad_norm(s["grads"], c["max_norm"], out=s["outs"]))
    recipe = fq.Recipe.MX_1x32_TILED if c["recipe"] == "mx" else fq.Recipe.TENSOR
    out = fq.OutDtype.FP32 if c["out"] == "fp32" else fq.OutDtype.BF16
    operands = (s["a"], fmt[c["fa"]], recipe, s["sa"], s["b"], fmt[c["fb"]], recipe, s["sb"], s["offsets"])
    if c["op"] == "group_wgrad":
        return {"dw": fq.grouped_wgrad(*operands, out=out)}
    return {"y": fq.grouped_gemm(*operands, out=out, stacked=fq.Stacked.ROWS if c["op"] == "group_fwd" else fq.Stacked.COLS)}


_PLAIN = {"rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd, "group_fwd": _product, "group_dgrad": _product, "group_wgrad": _product,
          "clip": _clip_norm}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"].startswith("rms"):
        n, e = c["rows"] * c["cols"], _SIZE[c["dtype"]]
        params = c["cols"] * _SIZE[c["wdtype"]]
        if c["op"] == "rms_bwd":
            return {"bytes": (4 if c["residual"] else 3) * n * e + 4 * c["rows"] + 2 * params, "flops": 9 * n}
        scales = {"": 0, "tensor": 8, "1x128": 4 * c["rows"] * -(-c["cols"] // 128)}.get(c["recipe"], n // 32)
        return {"bytes": n * e * (1 + 2 * c["residual"] + c["keep_y"]) + params + 4 * c["rows"] + (n if c["recipe"] else 0) + scales,
                "flops": 7 * n}
    if c["op"] == "clip":
        sizes = [int(v) for v in c["sizes"].split()]
        size = sum(n * (4 if c["dtype"] == "fp32" or c["dtype"] == "mixed" and i % 3 == 2 else 2) for i, n in enumerate(sizes))
        return {"bytes": 2 * size, "flops": 3 * sum(sizes)}
    rows, n, depth = c["tokens"] * c["k"], c["n"], c["depth"]
    used = min(rows, c["experts"])   # experts with rows
    flops = 2 * rows * n * depth
    scales = 33 / 32 if c["recipe"] == "mx" else 1
    if c["op"] == "group_wgrad":
        return {"bytes": rows * (n + depth) * scales + c["experts"] * n * depth * _SIZE[c["out"]], "flops": flops}
    return {"bytes": (rows + used * n) * depth * scales + _capacity(c) * n * _SIZE[c["out"]], "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_operand(codes, mult):
    v = codes.float().double()
    if mult.dtype == torch.float32:
        return v * mult.double()
    power = torch.exp2(mult.view(torch.uint8).double() - 127)
    atoms, (rows, cols) = power.view(-1, 512), codes.shape
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(cols // 32, device="cuda")[None]
    scale = atoms[(r // 128) * (cols // 128) + b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]
    return v * scale.repeat_interleave(32, 1)


def exact(case, seed):
    """The operators in 64 bits.  The 8-bit codes and power-of-two multipliers have no entry: which of two a value on their
    border takes is a matter of the working precision."""
    c, s = case, prepare(case, seed)
    if c["op"] == "rms_fwd":
        dt = _DT[c["dtype"]]
        h = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
        h = h.to(dt).double()
        rms = h.pow(2).mean(1).add(_EPS).rsqrt()
        y = torch.einsum("rc,r,c->rc", h, rms, s["weight"].double())
        out = {"rstd": rms}
        if c["residual"]:
            out["h"] = h
        if c["keep_y"]:
            out["y"] = y
        if c["recipe"]:
            out["codes"] = None
            if c["recipe"] == "tensor":
                out["amax"] = torch.linalg.vector_norm(y, math.inf).reshape(1)
            elif c["recipe"] == "1x128":
                amax = torch.stack([p.abs().amax(1) for p in y.split(128, 1)], 1)
                out["mult"] = torch.where(amax > 0, amax / _FMAX[c["fmt"]], 1.0)
            else:
                out["mult"] = None
        return out
    if c["op"] == "rms_bwd":
        h, r, dy, w = s["h"].double(), s["rstd"].double(), s["dy"].double(), s["weight"].double()
        # dx_i = r w_i dy_i - r^3 h_i / n sum_j w_j dy_j h_j
        dot = torch.einsum("rc,rc,c->r", dy, h, w)
        dx = torch.einsum("rc,c,r->rc", dy, w, r) - h * (r ** 3 * dot / c["cols"])[:, None]
        if c["residual"]:
            dx += s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", dy, h, r)}
    if c["op"] == "clip":
        total = math.sqrt(math.fsum(float(torch.dot(g.double(), g.double())) for g in s["grads"]))
        coef = min(1.0, c["max_norm"] / (total + 1e-6))
        return _clipped({**s, **{n + "_out": s[n].double() * coef for n in ("bf16", "fp32") if s[n] is not None}},
                        torch.tensor([total], dtype=torch.float64))
    starts, n, depth = s["offsets"].tolist(), c["n"], c["depth"]
    a = _exact_operand(s["a"], s["sa"])
    if c["op"] == "group_wgrad":
        b = _exact_operand(s["b"], s["sb"])
        return {"dw": torch.stack([torch.einsum("nr,dr->nd", a[:, lo:hi], b[:, lo:hi]) for lo, hi in zip(starts, starts[1:])])}
    b = _exact_operand(s["b"], s["sb"])
    y = torch.zeros(a.shape[0], n, dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        w = b[e * n:(e + 1) * n] if c["op"] == "group_fwd" else b[:, e * depth:(e + 1) * depth]
        y[starts[e]:starts[e + 1]] = torch.einsum("rd,nd->rn", a[starts[e]:starts[e + 1]], w)
    return {"y": y}
