"""Cases of the pre-norm FP8 feed-forward operators, with their plain forms.

Four operators that stand around the scaled-FP8 products of a transformer
block:

  norm       r = x + residual; y = r / rms(r) * w; FP8 codes of y with one
             scale per tensor (delayed scaling) or per 1x128 group
  norm_grad  its backward pass: dx (with the gradient that reaches the sum
             directly), dw, and the E5M2 codes of dx under a delayed scale
  gemm       y = act(sa sb A B^T + bias) + residual, with z = the argument of
             act kept for the backward pass and FP8 codes of y; operands with
             one scale per tensor, or 1x128 x 128x128 group scales
  act_grad   dz = (sa sb A B) * act'(z): the data gradient taken through the
             activation, its E5M2 codes and the bias gradient

``own`` False: ``run`` computes them with elementary torch operations in fp32,
rounded once at the end.  ``own`` True: ``run`` calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3, E5M2 = 0, 1
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
F8_MAX = (448.0, 57344.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "relu2", "silu", "gelu_tanh", "gelu")
EPS = 1e-5


def listed():
    return [
        # one token of a decoder layer: the norm ahead of a 1x128-group product
        dict(name="norm_token", op="norm", mode="group", sfmt="f32", m=1, k=7168, dt="bf16",
             wdt="bf16", res=True, inv=False),
        # a batch of decoded tokens with power-of-two group scales
        dict(name="norm_batch_ue8m0", op="norm", mode="group", sfmt="ue8m0", m=16, k=7168,
             dt="bf16", wdt="bf16", res=True, inv=False),
        # the norm of a training step: delayed per-tensor scale, 1/rms kept
        dict(name="norm_train", op="norm", mode="tensor", sfmt="f32", m=16384, k=4096, dt="bf16",
             wdt="f32", res=True, inv=True),
        # its backward pass
        dict(name="norm_grad_train", op="norm_grad", m=16384, k=4096, dt="bf16", dydt="bf16",
             wdt="f32", dres=True, codes=True),
        # a short ragged step in fp32, rows that fill no whole group
        dict(name="norm_grad_ragged", op="norm_grad", m=777, k=2064, dt="f32", dydt="f32",
             wdt="f32", dres=False, codes=False),
        # one token through a fine-grained down projection, added to the stream
        dict(name="group_token", op="gemm", mode="group", sfmt="f32", m=1, n=2048, k=7168,
             act="none", bias=True, res="bf16", pre=False, out="bf16", codes=False),
        # a prefill chunk through a fine-grained up projection
        dict(name="group_chunk", op="gemm", mode="group", sfmt="ue8m0", m=4096, n=7168, k=2048,
             act="silu", bias=True, res="", pre=False, out="bf16", codes=False),
        # odd sizes and an fp32 stream
        dict(name="tensor_ragged", op="gemm", mode="tensor", sfmt="f32", m=1000, n=2053, k=2064,
             act="relu2", bias=True, res="f32", pre=False, out="f32", codes=False),
        # up and down projections of a training step
        dict(name="up_train", op="gemm", mode="tensor", sfmt="f32", m=16384, n=14336, k=4096,
             act="gelu_tanh", bias=True, res="", pre=True, out="", codes=True),
        dict(name="down_train", op="gemm", mode="tensor", sfmt="f32", m=16384, n=4096, k=14336,
             act="none", bias=True, res="bf16", pre=False, out="bf16", codes=False),
        # the data gradient of the down projection, through the activation
        dict(name="act_grad_train", op="act_grad", m=16384, n=14336, k=4096, act="gelu_tanh",
             out="", codes=True, dbias=True),
        # a short ragged step, gradient stored in bf16 too
        dict(name="act_grad_ragged", op="act_grad", m=333, n=1040, k=528, act="gelu", out="bf16",
             codes=True, dbias=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "gemm", "gemm", "gemm", "act_grad"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("norm", "norm_grad"):
        k = _log(rng, 256, 16384, 16)
        m = min(_log(rng, 1, 16384), max(1, 16384 * 4096 // k))
        if op == "norm":
            mode = rng.choice(["tensor", "group"])
            # power-of-two scales round up: a last-bit difference doubles the
            # scale of a group at a boundary, so they are drawn for few rows
            sfmt = "ue8m0" if mode == "group" and m <= 64 and flag() else "f32"
            return dict(op=op, mode=mode, sfmt=sfmt, m=m, k=k, dt=rng.choice(["bf16", "bf16", "f32"]),
                        wdt=rng.choice(["bf16", "f32"]), res=flag(), inv=flag())
        return dict(op=op, m=m, k=k, dt=rng.choice(["bf16", "bf16", "f32"]),
                    dydt=rng.choice(["bf16", "f32"]), wdt=rng.choice(["bf16", "f32"]), dres=flag(),
                    codes=flag())
    if op == "gemm":
        mode = rng.choice(["tensor", "group"])
        m = _log(rng, 1, 16384)
        if mode == "group":
            k, n = _log(rng, 256, 8192, 128), _log(rng, 128, 8192)
            return dict(op=op, mode=mode, sfmt=rng.choice(["f32", "ue8m0"]), m=m, n=n, k=k,
                        act=rng.choice(ACTS), bias=flag(), res=rng.choice(["", "bf16"]),
                        pre=flag(), out="bf16", codes=False)
        k, n = _log(rng, 128, 14336, 16), _log(rng, 128, 14336, 16)
        if m * n * k > 16384 * 14336 * 4096:
            m = 16384 * 14336 * 4096 // (n * k)
        codes = flag()
        return dict(op=op, mode=mode, sfmt="f32", m=m, n=n, k=k, act=rng.choice(ACTS), bias=flag(),
                    res=rng.choice(["", "bf16", "f32"]), pre=flag(),
                    out=rng.choice(["", "bf16"]) if codes else rng.choice(["bf16", "f32"]),
                    codes=codes)
    k, n, m = _log(rng, 128, 8192, 16), _log(rng, 128, 14336, 16), _log(rng, 32, 16384)
    if m * n * k > 16384 * 14336 * 4096:
        m = 16384 * 14336 * 4096 // (n * k)
    codes = flag()
    return dict(op=op, m=m, n=n, k=k, act=rng.choice(ACTS[1:]),
                out="" if codes and flag() else "bf16", codes=codes, dbias=flag())


# ----------------------------------------------------------------- inputs --

def _randn(shape, std, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV).mul_(std).to(dtype)


def _stream(m, k, gen, dtype):
    """A residual stream: unit variance with a few loud columns."""
    x = torch.randn((m, k), generator=gen, device=DEV)
    loud = torch.randperm(k, generator=gen, device=DEV)[: max(1, k // 200)]
    x[:, loud] *= 20.0
    return x.to(dtype)


def _codes_tensor(shape, std, fmt, gen):
    """Codes of a normal tensor under its own amax, and the scale."""
    x = torch.randn(shape, generator=gen, device=DEV).mul_(std)
    s = (x.abs().amax() / F8_MAX[fmt]).reshape(1)
    return (x / s).clamp_(-F8_MAX[fmt], F8_MAX[fmt]).to(F8[fmt]).view(torch.uint8), s


def _pow2_up(s):
    """Exponent of the smallest power of two not below s."""
    man, e = torch.frexp(s)
    return torch.where(man == 0.5, e - 1, e)


def _group_scales(amax, sfmt):
    s = torch.where(amax > 0, amax / F8_MAX[0], torch.ones_like(amax))
    if sfmt == "f32":
        return s, s
    e = _pow2_up(s)
    return torch.ldexp(torch.ones_like(s), e), (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    c, st = case, {"case": dict(case)}
    m, k = c["m"], c["k"]
    n = c.get("n", 0)
    buf = lambda shape, dt: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
    u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
    if c["op"] == "norm":
        dt = TYPES[c["dt"]]
        st["x"] = _randn((m, k), 1.0, gen, dt) if c["res"] else _stream(m, k, gen, dt)
        st["residual"] = _stream(m, k, gen, dt) if c["res"] else None
        st["w"] = _randn((k,), 0.1, gen).add_(1.0).to(TYPES[c["wdt"]])
        st["sum"] = buf((m, k), dt) if c["res"] else None
        st["q"] = buf((m, k), u8)
        st["inv"] = buf((m,), f32) if c["inv"] else None
        g = (k + 127) // 128
        if c["mode"] == "tensor":
            st["scale"] = torch.full((1,), 12.0 / 448.0, device=DEV)
            st["amax"] = buf((1,), f32)
        else:
            st["scales"] = buf((g, m), f32 if c["sfmt"] == "f32" else u8)
    elif c["op"] == "norm_grad":
        dt = TYPES[c["dt"]]
        st["dy"] = _randn((m, k), 1e-3, gen, TYPES[c["dydt"]])
        st["r"] = _stream(m, k, gen, dt)
        st["inv"] = torch.rsqrt(st["r"].float().square().mean(1) + EPS)
        st["w"] = _randn((k,), 0.1, gen).add_(1.0).to(TYPES[c["wdt"]])
        st["dres"] = _randn((m, k), 1e-3, gen, dt) if c["dres"] else None
        st["dx"], st["dw"] = buf((m, k), dt), buf((k,), f32)
        if c["codes"]:
            st["q"], st["amax"] = buf((m, k), u8), buf((1,), f32)
            st["scale"] = torch.full((1,), 6e-3 / 57344.0, device=DEV)
    elif c["op"] == "gemm":
        st["bias"] = _randn((n,), 0.5, gen) if c["bias"] else None
        st["residual"] = _stream(m, n, gen, TYPES[c["res"]]) if c["res"] else None
        st["out"] = buf((m, n), TYPES[c["out"]]) if c["out"] else None
        st["pre"] = buf((m, n), bf) if c["pre"] else None
        if c["mode"] == "tensor":
            st["a"], st["sa"] = _codes_tensor((m, k), 1.0, E4M3, gen)
            st["b"], st["sb"] = _codes_tensor((n, k), 1.3 / math.sqrt(k), E4M3, gen)
        else:
            g = k // 128
            x = _stream(m, k, gen, f32)
            s, st["sa"] = _group_scales(x.view(m, g, 128).abs().amax(2).t().contiguous(), c["sfmt"])
            q = x.view(m, g, 128) / s.t().unsqueeze(2)
            st["a"] = q.clamp_(-448, 448).to(F8[0]).view(u8).view(m, k)
            nb = (n + 127) // 128
            x = torch.zeros((nb * 128, k), device=DEV)
            x[:n] = _randn((n, k), 1.0 / math.sqrt(k), gen)
            s, st["sb"] = _group_scales(x.view(nb, 128, g, 128).abs().amax((1, 3)), c["sfmt"])
            q = x.view(nb, 128, g, 128) / s[:, None, :, None]
            st["b"] = q.clamp_(-448, 448).to(F8[0]).view(u8).view(nb * 128, k)[:n].contiguous()
        if c["codes"]:
            st["q"], st["amax"] = buf((m, n), u8), buf((1,), f32)
            st["scale"] = torch.full((1,), 8.0 / 448.0, device=DEV)
    else:
        st["a"], st["sa"] = _codes_tensor((m, k), 1e-3, E5M2, gen)
        # the down projection's weight [k, n], as the forward pass keeps it
        st["b"], st["sb"] = _codes_tensor((k, n), 1.0 / math.sqrt(n), E4M3, gen)
        st["pre"] = _randn((m, n), 1.3, gen, bf)
        st["out"] = buf((m, n), bf) if c["out"] else None
        st["dbias"] = buf((n,), f32) if c["dbias"] else None
        if c["codes"]:
            st["q"], st["amax"] = buf((m, n), u8), buf((1,), f32)
            st["scale"] = torch.full((1,), 8e-3 * math.sqrt(k / n) / 57344.0, device=DEV)
    return st


# ------------------------------------------------------------- plain form --

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "relu2":
        return z.clamp_min(0).square()
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2 * z.clamp_min(0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * (c * (1 + 3 * 0.044715 * z * z))
    if act == "gelu":
        return (0.5 * torch.erfc(z * -math.sqrt(0.5))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    return torch.ones_like(z)


def _cast(y, scale, fmt):
    return (y / scale).clamp(-F8_MAX[fmt], F8_MAX[fmt]).to(F8[fmt])


def _with(**kw):
    return {name: v for name, v in kw.items() if v is not None}


def _plain_norm(c, st):
    r = st["x"].float()
    if c["res"]:
        st["sum"].copy_(r + st["residual"].float())
        r = st["sum"].float()
    inv = torch.rsqrt(r.square().mean(1) + EPS)
    y = r * inv[:, None] * st["w"].float()
    out = _with(sum=st["sum"], inv=inv if c["inv"] else None)
    if c["mode"] == "tensor":
        return dict(out, q=_cast(y, st["scale"], E4M3), amax=y.abs().amax().reshape(1))
    m, k = y.shape
    g = (k + 127) // 128
    yp = torch.nn.functional.pad(y, (0, g * 128 - k)).view(m, g, 128)
    s, kept = _group_scales(yp.abs().amax(2), c["sfmt"])
    q = _cast(yp, s.unsqueeze(2), E4M3).view(m, g * 128)[:, :k].contiguous()
    kept = kept.t().contiguous()
    return dict(out, q=q, scales=kept if c["sfmt"] == "f32" else kept.view(torch.float8_e8m0fnu))


def _plain_norm_grad(c, st):
    dy, w, inv = st["dy"].float(), st["w"].float(), st["inv"][:, None]
    xhat = st["r"].float() * inv
    g = dy * w
    dx = inv * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if c["dres"]:
        dx = dx + st["dres"].float()
    out = dict(dx=dx.to(TYPES[c["dt"]]), dw=(dy * xhat).sum(0))
    if c["codes"]:
        out.update(q=_cast(dx, st["scale"], E5M2), amax=dx.abs().amax().reshape(1))
    return out


def _group_values(q, s, sfmt, rows, per):
    """fp32 values of group-scaled codes: s [groups of rows, K / 128]."""
    if sfmt == "ue8m0":
        s = torch.ldexp(torch.ones(s.shape, device=DEV), s.int() - 127)
    s = s.repeat_interleave(per, 0)[:rows] if per > 1 else s
    v = q.view(F8[0]).float()
    return (v.view(rows, -1, 128) * s.unsqueeze(2)).view(rows, -1)


def _plain_gemm(c, st):
    if c["mode"] == "tensor":
        z = st["a"].view(F8[0]).float() @ st["b"].view(F8[0]).float().t()
        z *= st["sa"] * st["sb"]
    else:
        a = _group_values(st["a"], st["sa"].t(), c["sfmt"], c["m"], 1)
        b = _group_values(st["b"], st["sb"], c["sfmt"], c["n"], 128)
        z = a @ b.t()
    if c["bias"]:
        z += st["bias"]
    y = _act(z, c["act"])
    if c["res"]:
        y = y + st["residual"].float()
    out = {}
    if c["pre"]:
        out["pre"] = z.to(torch.bfloat16)
    if c["out"]:
        out["out"] = y.to(TYPES[c["out"]])
    if c["codes"]:
        out.update(q=_cast(y, st["scale"], E4M3), amax=y.abs().amax().reshape(1))
    return out


def _plain_act_grad(c, st):
    dz = st["a"].view(F8[1]).float() @ st["b"].view(F8[0]).float()
    dz *= st["sa"] * st["sb"]
    dz *= _act_slope(st["pre"].float(), c["act"])
    out = {}
    if c["out"]:
        out["out"] = dz.to(torch.bfloat16)
    if c["codes"]:
        out.update(q=_cast(dz, st["scale"], E5M2), amax=dz.abs().amax().reshape(1))
    if c["dbias"]:
        out["dbias"] = dz.sum(0)
    return out


# ---------------------------------------------------------------- library --

def _own_norm(F, c, st):
    out = _with(sum=st["sum"], inv=st["inv"])
    if c["mode"] == "tensor":
        F.fp8_rmsnorm_quantize(st["x"], st["w"], EPS, F.E4M3, st["q"], residual=st["residual"],
                               sum_out=st["sum"], scale=st["scale"], amax_out=st["amax"],
                               inv_rms=st["inv"])
        return dict(out, q=st["q"].view(F8[0]), amax=st["amax"])
    f32 = c["sfmt"] == "f32"
    F.fp8_rmsnorm_quantize(st["x"], st["w"], EPS, F.E4M3, st["q"], residual=st["residual"],
                           sum_out=st["sum"], scales=st["scales"],
                           sfmt=F.SCALE_F32 if f32 else F.SCALE_UE8M0, inv_rms=st["inv"])
    return dict(out, q=st["q"].view(F8[0]),
                scales=st["scales"] if f32 else st["scales"].view(torch.float8_e8m0fnu))


def _own_norm_grad(F, c, st):
    out = dict(dx=st["dx"], dw=st["dw"])
    if c["codes"]:
        F.fp8_rmsnorm_backward(st["dy"], st["r"], st["inv"], st["w"], st["dx"],
                               d_residual=st["dres"], dw=st["dw"], q=st["q"], fmt=F.E5M2,
                               scale=st["scale"], amax_out=st["amax"])
        return dict(out, q=st["q"].view(F8[1]), amax=st["amax"])
    F.fp8_rmsnorm_backward(st["dy"], st["r"], st["inv"], st["w"], st["dx"],
                           d_residual=st["dres"], dw=st["dw"])
    return out


def _own_gemm(F, c, st):
    act = ACTS.index(c["act"])
    out = _with(pre=st["pre"], out=st["out"])
    if c["mode"] == "group":
        F.fp8_gemm_group_epilogue(st["a"], st["sa"], st["b"], st["sb"],
                                  F.SCALE_F32 if c["sfmt"] == "f32" else F.SCALE_UE8M0, st["out"],
                                  bias=st["bias"], act=act, residual=st["residual"],
                                  pre_out=st["pre"])
        return out
    if c["codes"]:
        F.fp8_gemm_tensor_epilogue(st["a"], F.E4M3, st["b"], F.E4M3, st["sa"], st["sb"],
                                   st["out"], bias=st["bias"], act=act, residual=st["residual"],
                                   pre_out=st["pre"], q=st["q"], q_fmt=F.E4M3,
                                   q_scale=st["scale"], q_amax=st["amax"])
        return dict(out, q=st["q"].view(F8[0]), amax=st["amax"])
    F.fp8_gemm_tensor_epilogue(st["a"], F.E4M3, st["b"], F.E4M3, st["sa"], st["sb"], st["out"],
                               bias=st["bias"], act=act, residual=st["residual"],
                               pre_out=st["pre"])
    return out


def _own_act_grad(F, c, st):
    out = _with(out=st["out"], dbias=st["dbias"])
    kw = {}
    if c["codes"]:
        kw = dict(q=st["q"], q_fmt=F.E5M2, q_scale=st["scale"], q_amax=st["amax"])
        out.update(q=st["q"].view(F8[1]), amax=st["amax"])
    F.fp8_gemm_tensor_act_backward(st["a"], F.E5M2, st["b"], F.E4M3, st["sa"], st["sb"],
                                   st["pre"], ACTS.index(c["act"]), out=st["out"],
                                   dbias=st["dbias"], b_layout=F.MN_MAJOR, **kw)
    return out


def run(state):
    c = state["case"]
    if own:
        import fp8_quantized_gemm_gb300 as F
        return {"norm": _own_norm, "norm_grad": _own_norm_grad, "gemm": _own_gemm,
                "act_grad": _own_act_grad}[c["op"]](F, c, state)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "gemm": _plain_gemm,
            "act_grad": _plain_act_grad}[c["op"]](c, state)


# ----------------------------------------------------------- floor and truth --

def work(case):
    c = case
    m, k, n = c["m"], c["k"], c.get("n", 0)
    size = {"bf16": 2, "f32": 4, "": 0}
    if c["op"] == "norm":
        e = size[c["dt"]]
        b = m * k * (e * (3 if c["res"] else 1) + 1) + k * size[c["wdt"]]
        b += 4 * m if c["inv"] else 0
        if c["mode"] == "group":
            b += (k + 127) // 128 * m * (4 if c["sfmt"] == "f32" else 1)
        return {"bytes": b, "flops": 8 * m * k}
    if c["op"] == "norm_grad":
        e = size[c["dt"]]
        b = m * k * (size[c["dydt"]] + e * (3 if c["dres"] else 2) + (1 if c["codes"] else 0))
        return {"bytes": b + 4 * m + k * (4 + size[c["wdt"]]), "flops": 10 * m * k}
    b = (m + n) * k + m * n * (size[c["out"]] + (1 if c["codes"] else 0))
    if c["op"] == "gemm":
        b += m * n * ((2 if c["pre"] else 0) + size[c["res"]]) + (4 * n if c["bias"] else 0)
        if c["mode"] == "group":
            e = 4 if c["sfmt"] == "f32" else 1
            b += e * (k // 128) * (m + (n + 127) // 128)
    else:
        b += 2 * m * n + (4 * n if c["dbias"] else 0)
    return {"bytes": b, "flops": 2.0 * m * n * k}


def exact(case, seed):
    """The definitions in 64 bits; codes as the unrounded quotients they stand
    for, within the format's range."""
    c, st = case, prepare(case, seed)
    d = lambda t: t.double()  # noqa: E731
    coded = lambda y, fmt: (y / d(st["scale"])).clamp(-F8_MAX[fmt], F8_MAX[fmt])  # noqa: E731
    phi = lambda z: 0.5 * (1 + torch.special.erf(z / math.sqrt(2)))  # noqa: E731
    if c["op"] == "norm":
        r = d(st["x"])
        out = {}
        if c["res"]:
            r = d((r + d(st["residual"])).to(TYPES[c["dt"]]))  # the stream is kept in its type
            out["sum"] = r
        rms = torch.sqrt(r.pow(2).sum(1, keepdim=True) / c["k"] + EPS)
        if c["inv"]:
            out["inv"] = (1 / rms).squeeze(1)
        y = d(st["w"]) * (r / rms)
        if c["mode"] == "tensor":
            return dict(out, q=coded(y, E4M3), amax=y.abs().max().reshape(1))
        parts = torch.split(y, 128, dim=1)
        tops = torch.stack([p.abs().amax(1) for p in parts])
        s = torch.where(tops > 0, tops / 448.0, torch.ones_like(tops))
        if c["sfmt"] == "ue8m0":
            s = torch.exp2(torch.ceil(torch.log2(s)))
        q = torch.cat([p / s[i][:, None] for i, p in enumerate(parts)], 1).clamp(-448, 448)
        return dict(out, q=q, scales=s)
    if c["op"] == "norm_grad":
        inv, r = d(st["inv"])[:, None], d(st["r"])
        g = d(st["dy"]) * d(st["w"])
        dot = (g * r).sum(1, keepdim=True)
        dx = g * inv - r * dot * inv.pow(3) / c["k"]
        if c["dres"]:
            dx = dx + d(st["dres"])
        out = dict(dx=dx, dw=(d(st["dy"]) * r * inv).sum(0))
        if c["codes"]:
            out.update(q=coded(dx, E5M2), amax=dx.abs().max().reshape(1))
        return out
    if c["op"] == "gemm":
        a, b = d(st["a"].view(F8[0]).float()), d(st["b"].view(F8[0]).float())
        if c["mode"] == "tensor":
            z = torch.matmul(a, b.T) * (d(st["sa"]) * d(st["sb"]))
        else:
            value = (lambda s: d(s)) if c["sfmt"] == "f32" else (lambda s: torch.exp2(d(s) - 127))
            sa, sb = value(st["sa"]), value(st["sb"])
            for g in range(c["k"] // 128):
                a[:, 128 * g:128 * g + 128] *= sa[g][:, None]
                b[:, 128 * g:128 * g + 128] *= sb[:, g].repeat_interleave(128)[:c["n"], None]
            z = torch.matmul(a, b.T)
        del a, b
        if c["bias"]:
            z = z + d(st["bias"])
        y = {"none": lambda v: v, "relu": torch.relu, "relu2": lambda v: torch.relu(v) ** 2,
             "silu": lambda v: v * torch.sigmoid(v), "gelu": lambda v: v * phi(v),
             "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh(
                 math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))}[c["act"]](z)
        if c["res"]:
            y = y + d(st["residual"])
        out = _with(pre=z if c["pre"] else None, out=y if c["out"] else None)
        if c["codes"]:
            out.update(q=coded(y, E4M3), amax=y.abs().max().reshape(1))
        return out
    dz = torch.matmul(d(st["a"].view(F8[1]).float()), d(st["b"].view(F8[0]).float()))
    dz *= d(st["sa"]) * d(st["sb"])
    z = d(st["pre"])
    if c["act"] == "gelu":
        slope = phi(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    elif c["act"] == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        slope = 0.5 * (1 + t) + 0.5 * z * (1 - t ** 2) * a * (1 + 0.134145 * z ** 2)
    elif c["act"] == "silu":
        slope = torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    else:
        slope = torch.where(z > 0, 2 * z if c["act"] == "relu2" else torch.ones_like(z),
                            torch.zeros_like(z))
    dz *= slope
    out = {"out": dz} if c["out"] else {}
    if c["codes"]:
        out.update(q=coded(dz, E5M2), amax=dz.abs().max().reshape(1))
    if c["dbias"]:
        out["dbias"] = dz.sum(0)
    return out
