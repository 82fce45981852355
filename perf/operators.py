"""Cases that measure the linear-layer and row-norm operators.

Four operators around one projection of a transformer block, and what they
compute (T: the 16-bit type of the tensors, or fp32 where a case says so):

linear        z = alpha * scale_a[m] * scale_b[n] * (A . B^T) + bias[n],
              D = act(z) + residual, optionally Z = z kept for training
linear_grad   dZ = dD * act'(Z), dA = dZ . B, dB = dB_in + dZ^T . A,
              dbias = sum over rows of dZ
rmsnorm       h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, in 16
              bits or in 8 bits with one scale per row (amax / 448 for e4m3,
              amax / 127 for int8); H = h when there is a residual
rmsnorm_grad  with s = 1 / sqrt(mean(h^2) + eps) and g = dY * weight:
              dH = dH_in + s * g - h * s^3 * mean(g * h),
              dweight = sum over rows of dY * h * s

A is M x K, B (the weight) N x K, both with K contiguous; D, Z, residual and
dD are M x N.  ``own`` picks the framework's calls or the plain form.
"""
import math

import torch

own = False

EPS = 1e-6
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1, "i8": 1}
QMAX = {"e4m3": 448.0, "i8": 127.0}
PAD = 64  # elements between rows of a strided tensor, beyond the row itself


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _linear(name, M, N, K, ab, d, act="none", bias=True, res=False, z=False, pad=False, alpha=1.0):
    c = dict(op="linear", M=M, N=N, K=K, ab=ab, d=d, act=act, bias=bias, res=res, z=z, pad=pad, alpha=alpha)
    return dict(name=name, **c) if name else c


def _linear_grad(name, M, N, K, ab, db, act="none", db_in=False):
    c = dict(op="linear_grad", M=M, N=N, K=K, ab=ab, db=db, act=act, db_in=db_in)
    return dict(name=name, **c) if name else c


def _rmsnorm(name, rows, cols, x, y, res=True, pad=False):
    c = dict(op="rmsnorm", rows=rows, cols=cols, x=x, y=y, res=res, pad=pad)
    return dict(name=name, **c) if name else c


def _rmsnorm_grad(name, rows, cols, x, dh_in=True):
    c = dict(op="rmsnorm_grad", rows=rows, cols=cols, x=x, dh_in=dh_in)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token through an output projection: the weight's bytes and latency
        _linear("linear_token_bf16", 1, 4096, 4096, "bf16", "bf16", res=True),
        # sixteen sequences decoding with 8-bit weights and activations
        _linear("linear_decode16_e4m3", 16, 8192, 8192, "e4m3", "bf16", act="silu", bias=False),
        # training forward of an up projection: the pre-activation is kept
        _linear("linear_train_bf16", 4096, 4096, 4096, "bf16", "bf16", act="gelu", z=True),
        # a prefill in 8 bits, the largest product
        _linear("linear_prefill_e4m3", 8192, 8192, 8192, "e4m3", "bf16", res=True),
        # ragged sizes in strided buffers
        _linear("linear_ragged_f16", 1001, 2552, 4104, "f16", "f16", act="gelu_tanh", res=True, pad=True),
        # int8 serving at a medium batch
        _linear("linear_i8", 2048, 4096, 4096, "i8", "bf16", act="relu"),
        # backward of the training forward above
        _linear_grad("linear_grad_bf16", 4096, 4096, 4096, "bf16", "bf16", act="gelu"),
        # ragged backward of a plain projection, weight gradient added up in fp32
        _linear_grad("linear_grad_ragged_f16", 1001, 1032, 2568, "f16", "f32", db_in=True),
        # one token's norm in front of an 8-bit projection
        _rmsnorm("rmsnorm_token", 1, 4096, "bf16", "e4m3"),
        # the norm of a long prefill, read and written once
        _rmsnorm("rmsnorm_prefill", 8192, 8192, "bf16", "e4m3"),
        # training backward of the norm
        _rmsnorm_grad("rmsnorm_grad_bf16", 8192, 4096, "bf16"),
        # odd sizes: rows that are no multiple of anything
        _rmsnorm_grad("rmsnorm_grad_odd_f16", 333, 1001, "f16", dh_in=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step - 1)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "rmsnorm", "rmsnorm_grad"))
    if op == "linear":
        ab, d = rng.choice((("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32"),
                            ("e4m3", "bf16"), ("e4m3", "f32"), ("i8", "bf16"), ("i8", "f16")))
        return _linear("", _log(rng, 1, 8192), _log(rng, 256, 8192, 8), _log(rng, 256, 8192, 16), ab, d,
                       act=rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), bias=rng.random() < 0.7,
                       res=rng.random() < 0.5, z=rng.random() < 0.3, pad=rng.random() < 0.3,
                       alpha=rng.choice((1.0, 0.5)))
    if op == "linear_grad":
        act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
        ab = rng.choice(("bf16", "f16"))
        db = rng.choice((ab, "f32")) if act in ("none", "relu") else ab
        return _linear_grad("", _log(rng, 1, 8192), _log(rng, 256, 4096, 8), _log(rng, 256, 4096, 8), ab, db,
                            act=act, db_in=db == "f32" and rng.random() < 0.5)
    cols = _log(rng, 64, 16384)
    rows = _log(rng, 1, min(16384, (8192 * 8192) // cols))
    if op == "rmsnorm":
        x = rng.choice(("bf16", "f16", "f32"))
        return _rmsnorm("", rows, cols, x, rng.choice((x, "e4m3", "i8")), res=rng.random() < 0.6,
                        pad=rng.random() < 0.3)
    return _rmsnorm_grad("", rows, cols, rng.choice(("bf16", "f16", "f32")), dh_in=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
class _Draws:
    """Seeded normal draws on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, scale=1.0):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=torch.float32).mul_(scale)


def _strided(t, pad):
    """t itself, or a copy whose rows lie PAD elements further apart."""
    if not pad:
        return t
    big = torch.zeros(t.shape[0], t.shape[1] + PAD, dtype=torch.uint8 if t.dtype == TORCH["e4m3"] else t.dtype,
                      device="cuda").view(t.dtype)
    v = big[:, :t.shape[1]]
    if t.dtype == TORCH["e4m3"]:
        v.view(torch.uint8).copy_(t.view(torch.uint8))
    else:
        v.copy_(t)
    return v


def _empty(rows, cols, dtype, pad):
    return torch.empty(rows, cols + (PAD if pad else 0), dtype=TORCH[dtype], device="cuda")[:, :cols]


def _rows_to_8_bits(t, kind):
    """A row-wise 8-bit form of t: the values and one scale per row."""
    scale = (t.abs().amax(dim=1) / QMAX[kind]).clamp_min(2.0 ** -100)
    q = t / scale[:, None]
    return (q.round() if kind == "i8" else q).to(TORCH[kind]), scale


def prepare(case, seed):
    c, r = case, _Draws(seed)
    s = {"case": c}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        # activations behind a norm: channels of different weight
        a = r.normal(M, K) * torch.exp(r.normal(1, K, scale=0.3))
        b = r.normal(N, K, scale=K ** -0.5)
        if c["ab"] in QMAX:
            a, s["scale_a"] = _rows_to_8_bits(a, c["ab"])
            b, s["scale_b"] = _rows_to_8_bits(b, c["ab"])
        else:
            a, b = a.to(TORCH[c["ab"]]), b.to(TORCH[c["ab"]])
        s["A"], s["B"] = _strided(a, c["pad"]), b
        if c["bias"]:
            s["bias"] = r.normal(N, scale=0.2)
        if c["res"]:
            s["residual"] = _strided(r.normal(M, N).to(TORCH[c["d"]]), c["pad"])
        s["D"] = _empty(M, N, c["d"], c["pad"])
        if c["z"]:
            s["Z"] = _empty(M, N, c["d"], False)
    elif c["op"] == "linear_grad":
        M, N, K, T = c["M"], c["N"], c["K"], TORCH[c["ab"]]
        s["dD"] = r.normal(M, N).to(T)
        s["A"] = r.normal(M, K).to(T)
        s["B"] = r.normal(N, K, scale=K ** -0.5).to(T)
        if c["act"] != "none":
            s["Z"] = r.normal(M, N).to(T)
            s["dZ"] = torch.empty(M, N, dtype=T, device="cuda")
        if c["db_in"]:
            s["dB_in"] = r.normal(N, K, scale=M ** 0.5)
        s["dA"] = torch.empty(M, K, dtype=T, device="cuda")
        s["dB"] = torch.empty(N, K, dtype=TORCH[c["db"]], device="cuda")
        s["dbias"] = torch.empty(N, dtype=torch.float32, device="cuda")
    else:
        R, C, T = c["rows"], c["cols"], TORCH[c["x"]]
        # a residual stream: some channels far larger than the rest
        chan = torch.exp(r.normal(1, C, scale=0.7))
        s["weight"] = (1.0 + r.normal(C, scale=0.2)).to(T)
        if c["op"] == "rmsnorm":
            s["x"] = _strided((r.normal(R, C) * chan).to(T), c["pad"])
            if c["res"]:
                s["residual"] = _strided((r.normal(R, C) * chan).to(T), c["pad"])
                s["H"] = _empty(R, C, c["x"], c["pad"])
            s["Y"] = _empty(R, C, c["y"], False)
            if c["y"] in QMAX:
                s["scale"] = torch.empty(R, dtype=torch.float32, device="cuda")
        else:
            s["H"] = (r.normal(R, C) * chan).to(T)
            s["dY"] = r.normal(R, C).to(T)
            if c["dh_in"]:
                s["dH_in"] = r.normal(R, C).to(T)
            s["dH"] = torch.empty(R, C, dtype=T, device="cuda")
            s["dweight"] = torch.empty(C, dtype=torch.float32, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
_plans = {}  # a program keeps one plan per problem shape


def _plan(c):
    key = tuple(sorted((k, v) for k, v in c.items() if k != "name"))
    if key not in _plans:
        import beta_epilogue_amd as be
        if c["op"] == "linear":
            _plans[key] = be.FusedLinear(
                c["M"], c["N"], c["K"], ab=c["ab"], d=c["d"], act=c["act"], bias="f32" if c["bias"] else None,
                residual=c["res"], z=c["z"], scale_a=c["ab"] in QMAX, scale_b=c["ab"] in QMAX,
                lda=c["K"] + PAD if c["pad"] else 0, ldd=c["N"] + PAD if c["pad"] else 0,
                ldr=c["N"] + PAD if c["pad"] and c["res"] else 0)
        elif c["op"] == "linear_grad":
            _plans[key] = be.FusedLinearGrad(c["M"], c["N"], c["K"], ab=c["ab"], act=c["act"], da=c["ab"],
                                             db=c["db"], dbias="f32")
        elif c["op"] == "rmsnorm":
            ld = c["cols"] + PAD if c["pad"] else 0
            _plans[key] = be.RmsNorm(c["rows"], c["cols"], x=c["x"], y=c["y"], weight=c["x"], residual=c["res"],
                                     eps=EPS, ldx=ld, ldr=ld if c["res"] else 0, ldh=ld if c["res"] else 0)
        else:
            _plans[key] = be.RmsNormGrad(c["rows"], c["cols"], x=c["x"], weight=c["x"], dweight="f32", eps=EPS)
    return _plans[key]


def _own(s):
    c, op = s["case"], _plan(s["case"])
    if c["op"] == "linear":
        op(s["A"], s["B"], bias=s.get("bias"), scale_a=s.get("scale_a"), scale_b=s.get("scale_b"),
           residual=s.get("residual"), D=s["D"], Z=s.get("Z"), alpha=c["alpha"])
        return {k: s[k] for k in ("D", "Z") if k in s}
    if c["op"] == "linear_grad":
        op(s["dD"], s["A"], s["B"], Z=s.get("Z"), dB_in=s.get("dB_in"), dZ=s.get("dZ"), dA=s["dA"], dB=s["dB"],
           dbias=s["dbias"])
        return {k: s[k] for k in ("dZ", "dA", "dB", "dbias") if k in s}
    if c["op"] == "rmsnorm":
        op(s["x"], s["weight"], residual=s.get("residual"), Y=s["Y"], H=s.get("H"), scale=s.get("scale"))
        return {k: _values(s[k]) for k in ("Y", "H", "scale") if k in s}
    op(s["dY"], s["H"], s["weight"], dH_in=s.get("dH_in"), dH=s["dH"], dweight=s["dweight"])
    return {"dH": s["dH"], "dweight": s["dweight"]}


def _values(t):
    """int8 as the numbers it stands for (every one is an fp16 value)."""
    return t.to(torch.float16) if t.dtype == torch.int8 else t


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.where(z <= 0, torch.zeros_like(z), z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 0.134145 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        T = TORCH[c["d"]]
        z = torch.mm(s["A"].float(), s["B"].float().t())
        if c["alpha"] != 1.0:
            z = z * c["alpha"]
        if "scale_a" in s:
            z = z * s["scale_a"][:, None] * s["scale_b"]
        if c["bias"]:
            z = z + s["bias"]
        d = _act(z, c["act"])
        if c["res"]:
            d = d + s["residual"].float()
        return {"D": d.to(T), "Z": z.to(T)} if c["z"] else {"D": d.to(T)}
    if c["op"] == "linear_grad":
        T = TORCH[c["ab"]]
        dz = s["dD"].float()
        if c["act"] != "none":
            dz = dz * _act_slope(s["Z"].float(), c["act"])
        db = torch.mm(dz.t(), s["A"].float())
        if c["db_in"]:
            db = db + s["dB_in"]
        out = {"dA": torch.mm(dz, s["B"].float()).to(T), "dB": db.to(TORCH[c["db"]]), "dbias": dz.sum(dim=0)}
        if c["act"] != "none":
            out["dZ"] = dz.to(T)
        return out
    w = s["weight"].float()
    if c["op"] == "rmsnorm":
        h = s["x"].float()
        out = {}
        if c["res"]:
            h = h + s["residual"].float()
            out["H"] = h.to(TORCH[c["x"]])
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * w
        if c["y"] in QMAX:
            out["scale"] = (y.abs().amax(dim=1) / QMAX[c["y"]]).clamp_min(2.0 ** -126)
            y = y / out["scale"][:, None]
            y = (y.round() if c["y"] == "i8" else y).clamp(-QMAX[c["y"]], QMAX[c["y"]])
        out["Y"] = _values(y.to(TORCH[c["y"]]))
        return out
    h, dy = s["H"].float(), s["dY"].float()
    rs = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    g = dy * w
    dh = rs * g - h * (rs * rs * rs * (g * h).mean(dim=1, keepdim=True))
    if c["dh_in"]:
        dh = dh + s["dH_in"].float()
    return {"dH": dh.to(TORCH[c["x"]]), "dweight": (dy * h * rs).sum(dim=0)}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K, es, ds = c["M"], c["N"], c["K"], SIZE[c["ab"]], SIZE[c["d"]]
        n = (M + N) * K * es + M * N * ds * (1 + c["res"] + c["z"]) + (4 * N if c["bias"] else 0)
        return {"bytes": n + (4 * (M + N) if c["ab"] in QMAX else 0), "flops": 2 * M * N * K}
    if c["op"] == "linear_grad":
        M, N, K, es = c["M"], c["N"], c["K"], SIZE[c["ab"]]
        n = es * (M * N * (3 if c["act"] != "none" else 1) + 2 * M * K + N * K) + 4 * N
        return {"bytes": n + N * K * SIZE[c["db"]] * (1 + c["db_in"]), "flops": 4 * M * N * K}
    R, C, xs = c["rows"], c["cols"], SIZE[c["x"]]
    if c["op"] == "rmsnorm":
        n = R * C * (xs * (3 if c["res"] else 1) + SIZE[c["y"]]) + C * xs
        return {"bytes": n + (4 * R if c["y"] in QMAX else 0), "flops": 6 * R * C}
    return {"bytes": R * C * xs * (4 if c["dh_in"] else 3) + C * (xs + 4), "flops": 12 * R * C}


def exact(case, seed):
    """The definition in 64 bits.  An 8-bit e4m3 result is given as the
    number that was to be rounded; int8 results have no such value."""
    c, s = case, prepare(case, seed)
    f = {k: v.to(torch.float32).to(torch.float64) for k, v in s.items() if torch.is_tensor(v)}
    half = math.sqrt(0.5)
    norm = math.sqrt(2.0 / math.pi)
    if c["op"] == "linear":
        z = c["alpha"] * (f["A"] @ f["B"].T)
        if c["ab"] in QMAX:
            z = torch.outer(f["scale_a"], f["scale_b"]) * z
        if c["bias"]:
            z = z + f["bias"][None, :]
        act = c["act"]
        if act == "relu":
            d = z.clamp_min(0.0)
        elif act == "gelu":
            d = z * torch.special.ndtr(z)
        elif act == "gelu_tanh":
            d = z * torch.sigmoid(2.0 * norm * (z + 0.044715 * z ** 3))
        elif act == "silu":
            d = z * torch.sigmoid(z)
        else:
            d = z
        out = {"D": d + f["residual"] if c["res"] else d}
        if c["z"]:
            out["Z"] = z
        return out
    if c["op"] == "linear_grad":
        dz, act = f["dD"], c["act"]
        if act != "none":
            z = f["Z"]
            if act == "relu":
                slope = torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
            elif act == "gelu":
                slope = torch.special.ndtr(z) + z * torch.exp(-(half * z) ** 2) / math.sqrt(2.0 * math.pi)
            elif act == "gelu_tanh":
                p = torch.sigmoid(2.0 * norm * (z + 0.044715 * z ** 3))
                slope = p + z * p * (1.0 - p) * 2.0 * norm * (1.0 + 3.0 * 0.044715 * z ** 2)
            else:
                p = torch.sigmoid(z)
                slope = p + z * p * (1.0 - p)
            dz = dz * slope
        db = dz.T @ f["A"]
        out = {"dA": dz @ f["B"], "dB": db + f["dB_in"] if c["db_in"] else db, "dbias": dz.sum(0)}
        if act != "none":
            out["dZ"] = dz
        return out
    if c["op"] == "rmsnorm":
        h = f["x"] + f["residual"] if c["res"] else f["x"]
        y = h / torch.sqrt(torch.mean(h ** 2, 1, keepdim=True) + EPS) * f["weight"]
        out = {"H": h} if c["res"] else {}
        if c["y"] in QMAX:
            out["scale"] = torch.amax(torch.abs(y), 1) / QMAX[c["y"]]
            out["Y"] = y / out["scale"][:, None] if c["y"] == "e4m3" else None
        else:
            out["Y"] = y
        return out
    h, g = f["H"], f["dY"] * f["weight"]
    r = torch.sqrt(torch.mean(h ** 2, 1, keepdim=True) + EPS)
    xhat = h / r
    dh = (g - xhat * torch.mean(g * xhat, 1, keepdim=True)) / r
    return {"dH": dh + f["dH_in"] if c["dh_in"] else dh, "dweight": (f["dY"] * xhat).sum(0)}
