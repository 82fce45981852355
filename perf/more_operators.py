"""Cases that measure the operators on rows that meet different weights: the
experts' and the adapters' of one batch.

T tokens choose top_k of E experts each (an id outside 0 .. E - 1: none, as
for padding); R = T * top_k rows lie sorted by expert, those of expert e at
offsets[e] .. offsets[e + 1] - 1, and rows past offsets[E] are left as they are.

expert_sort         offsets, rows[t][j] = the row of token t's j-th choice (-1:
                    none; within an expert the choices keep their order), and
                    Y[rows[t][j]] = X[t], 8 bits with a scale per row
expert_combine      D[t] = residual[t] + sum_j weights[t][j] Y[rows[t][j]]; without
                    weights and residual the gradient of the sort
   back             dY[rows[t][j]] = weights[t][j] dD[t],
                    dweights[t][j] = dD[t] . Y[rows[t][j]]
expert_linear       z = scale_a[r] scale_b[e][n] A[r] . B[e][n] + bias[e][n],
                    D = act(z) * U, optionally Z = z kept for training
expert_linear_grad  g = dD * U, dZ = g act'(Z), dU = dD act(Z), dA = dZ . B[e],
                    dB[e] = dB_in[e] + dZ^T . A, dbias[e] = sum of dZ, over e's rows
adapter_linear      D = act(A . B^T + bias + scale[g] (A . down[g]^T) . up[g]^T)
                    + residual, g = ids[m] (outside 0 .. G - 1: no adapter)

``own`` picks the framework's calls or the plain form.
"""
import math

import torch

own = False

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1, "i8": 1}
QMAX = {"e4m3": 448.0, "i8": 127.0}
PAD = 64  # elements between rows of a strided tensor, beyond the row itself


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _named(name, c):
    return dict(name=name, **c) if name else c


def _sort(name, T, k, E, cols, x, ids="i64", empty=0):
    return _named(name, dict(op="expert_sort", T=T, k=k, E=E, cols=cols, x=x, ids=ids, empty=empty))


def _combine(name, T, k, E, cols, x, weights=True, res=False, back=False, empty=0):
    return _named(name, dict(op="expert_combine", T=T, k=k, E=E, cols=cols, x=x, weights=weights, res=res, back=back,
                             empty=empty))


def _linear(name, T, k, E, N, K, ab, d, act="none", bias=False, mul=False, z=False, pad=False, empty=0):
    return _named(name, dict(op="expert_linear", T=T, k=k, E=E, N=N, K=K, ab=ab, d=d, act=act, bias=bias, mul=mul,
                             z=z, pad=pad, empty=empty))


def _linear_grad(name, T, k, E, N, K, ab, db, act="none", mul=False, db_in=False, empty=0):
    return _named(name, dict(op="expert_linear_grad", T=T, k=k, E=E, N=N, K=K, ab=ab, db=db, act=act, mul=mul,
                             db_in=db_in, empty=empty))


def _adapter(name, M, N, K, r, G, ab, runs, act="none", bias=False, res=False, pad=False):
    return _named(name, dict(op="adapter_linear", M=M, N=N, K=K, r=r, G=G, ab=ab, runs=runs, act=act, bias=bias,
                             res=res, pad=pad))


def listed():
    return [
        # sixteen sequences decoding: a call's latency
        _sort("sort_decode_bf16", 16, 8, 64, 2048, "bf16"),
        # a long prefill in 8 bits behind the norm, its last tokens padding
        _sort("sort_prefill_e4m3", 12345, 8, 128, 4096, "e4m3", ids="i32", empty=57),
        # the experts' results of that prefill back on the residual stream
        _combine("combine_prefill_bf16", 12345, 8, 128, 2048, "bf16", res=True, empty=57),
        # the gradient of a small odd sort
        _combine("sort_grad_odd_f16", 1001, 3, 13, 1032, "f16", weights=False),
        # training backward of the way back
        _combine("combine_grad_bf16", 8192, 2, 8, 4096, "bf16", back=True),
        # one token through its experts' gated projections: the weights' bytes
        _linear("experts_token_bf16", 1, 8, 64, 1536, 2048, "bf16", "bf16", act="silu", mul=True),
        # a serving batch with 8-bit weights, a few dozen rows for each expert
        _linear("experts_batch_e4m3", 256, 8, 64, 1536, 2048, "e4m3", "bf16"),
        # training forward of a gated projection, two of eight experts for each token
        _linear("experts_train_bf16", 8192, 2, 8, 4096, 2048, "bf16", "bf16", act="silu", mul=True, z=True),
        # its backward
        _linear_grad("experts_grad_bf16", 8192, 2, 8, 4096, 2048, "bf16", "bf16", act="silu", mul=True),
        # ragged backward of a plain projection, weight gradients added up in fp32
        _linear_grad("experts_grad_ragged_f16", 1001, 3, 13, 520, 1032, "f16", "f32", db_in=True, empty=17),
        # sixteen requests decoding, each with one of twelve adapters or none
        _adapter("adapters_decode16_bf16", 16, 4096, 4096, 16, 12, "bf16", runs=False),
        # the prompts of several requests packed into one batch
        _adapter("adapters_prefill_f16", 4001, 4096, 4096, 64, 7, "f16", runs=True, bias=True, res=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step - 1)))
    return min(hi, max(lo, int(v) // step * step))


def _tokens(rng, most):
    """Tokens, choices of each and experts: at most `most` rows."""
    E = _log(rng, 4, 160)
    k = rng.choice((1, 2, 3, 4, 6, 8))
    k = min(k, E)
    T = _log(rng, 1, most // k)
    return T, k, E, rng.choice((0, 0, min(T - 1, 5), T // 3))


def draw(rng):
    op = rng.choice(("expert_sort", "expert_combine", "expert_linear", "expert_linear", "expert_linear_grad",
                     "adapter_linear", "adapter_linear"))
    acts = ("none", "relu", "gelu", "gelu_tanh", "silu")
    if op == "expert_sort":
        x = rng.choice(("bf16", "f16", "f32", "e4m3", "i8"))
        cols = _log(rng, 256, 8192, 16)
        T, k, E, empty = _tokens(rng, min(131072, 12345 * 8 * 4096 // (cols * SIZE[x])))
        return _sort("", T, k, E, cols, x, ids=rng.choice(("i64", "i32")), empty=empty)
    if op == "expert_combine":
        x = rng.choice(("bf16", "f16", "f32"))
        cols = _log(rng, 256, 8192, 8)
        T, k, E, empty = _tokens(rng, 8192 * 4096 // cols)
        way = rng.choice(("weights", "weights", "sum", "back"))
        return _combine("", T, k, E, cols, x, weights=way != "sum", res=way != "back" and rng.random() < 0.5,
                        back=way == "back", empty=empty)
    if op == "adapter_linear":
        ab = rng.choice(("bf16", "f16"))
        return _adapter("", _log(rng, 1, 8192), _log(rng, 256, 4096, 8), _log(rng, 256, 4096, 8),
                        rng.choice((8, 16, 24, 32, 64)), _log(rng, 1, 48), ab, rng.random() < 0.5,
                        act=rng.choice(("none", "none", "silu", "gelu")), bias=rng.random() < 0.5,
                        res=rng.random() < 0.5, pad=rng.random() < 0.3)
    T, k, E, empty = _tokens(rng, 16384)
    K = _log(rng, 256, 4096, 16)
    N = _log(rng, 256, min(4096, max(256, 200000000 // (E * K)), max(256, 8192 * 2 * 4096 * 2048 // (T * k * K))), 8)
    act = rng.choice(acts)
    if op == "expert_linear":
        ab, d = rng.choice((("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"),
                            ("i8", "bf16"), ("i8", "f16")))
        return _linear("", T, k, E, N, K, ab, d, act=act, bias=rng.random() < 0.4, mul=rng.random() < 0.4,
                       z=rng.random() < 0.3, pad=rng.random() < 0.3, empty=empty)
    ab = rng.choice(("bf16", "f16"))
    plain = act in ("none", "relu")
    mul = not plain and rng.random() < 0.5
    db = rng.choice((ab, "f32")) if plain else ab
    return _linear_grad("", T, k, E, N, K, ab, db, act=act, mul=mul, db_in=db == "f32" and rng.random() < 0.5,
                        empty=empty)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
class _Draws:
    """Seeded draws on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, scale=1.0):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=torch.float32).mul_(scale)

    def whole(self, below, *shape):
        return torch.randint(0, below, shape, generator=self.g, device="cuda")


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


def _zeros(rows, cols, dtype, pad=False):
    n = cols + (PAD if pad else 0)
    if dtype == "e4m3":
        return torch.zeros(rows, n, dtype=torch.uint8, device="cuda").view(TORCH[dtype])[:, :cols]
    return torch.zeros(rows, n, dtype=TORCH[dtype], device="cuda")[:, :cols]


def _to_8_bits(t, kind):
    """An 8-bit form of t with one scale per row (of the last axis)."""
    scale = (t.abs().amax(dim=-1) / QMAX[kind]).clamp_min(2.0 ** -100)
    q = t / scale[..., None]
    return (q.round() if kind == "i8" else q).to(TORCH[kind]), scale


def _choices(r, c):
    """What a router gives: each token's experts, some of them favourites, and
    their weights; the last `empty` tokens have none."""
    logits = r.normal(c["T"], c["E"]) + r.normal(1, c["E"], scale=0.5)
    v, ids = torch.topk(logits, c["k"], dim=1)
    if c["empty"]:
        ids[c["T"] - c["empty"]:] = -1
    return ids, torch.softmax(v, dim=1)


def _offsets(ids, E):
    """Where each expert's rows begin, and the longest group's rows."""
    n = torch.bincount(ids[ids >= 0].reshape(-1), minlength=E)
    return torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32), max(1, int(n.max()))


def _rows(ids, E):
    """Each choice's row."""
    flat = ids.reshape(-1)
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device="cuda")
    return torch.where(flat < 0, -1, rows).to(torch.int32).reshape(ids.shape)


def prepare(case, seed):
    c, r = case, _Draws(seed)
    s = {"case": c}
    if c["op"] == "adapter_linear":
        M, N, K, G, T = c["M"], c["N"], c["K"], c["G"], TORCH[c["ab"]]
        s["A"] = _strided((r.normal(M, K) * torch.exp(r.normal(1, K, scale=0.3))).to(T), c["pad"])
        s["B"] = r.normal(N, K, scale=K ** -0.5).to(T)
        # one request in G + 1 has no adapter; a prompt's rows follow one another
        ids = r.whole(G + 1, M) - 1
        if c["runs"]:
            ids = ids[torch.sort(r.whole(max(1, min(M, 8)), M)).values]
        s["ids"] = ids.to(torch.int32)
        s["down"] = r.normal(G, c["r"], K, scale=K ** -0.5).to(T)
        s["up"] = r.normal(G, N, c["r"], scale=c["r"] ** -0.5).to(T)
        s["scale"] = torch.exp(r.normal(G, scale=0.3)) * 0.5
        if c["bias"]:
            s["bias"] = r.normal(N, scale=0.2)
        if c["res"]:
            s["residual"] = r.normal(M, N).to(T)
        s["D"] = _zeros(M, N, c["ab"], c["pad"])
        return s
    ids, weights = _choices(r, c)
    T, k, E = c["T"], c["k"], c["E"]
    R = T * k
    if c["op"] == "expert_sort":
        s["ids"] = ids if c["ids"] == "i64" else ids.to(torch.int32)
        x = r.normal(T, c["cols"])
        if c["x"] in QMAX:
            x, s["scale"] = _to_8_bits(x, c["x"])
            s["scale_out"] = torch.zeros(R, device="cuda")
        s["X"] = x.to(TORCH[c["x"]])
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["rows"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        s["Y"] = _zeros(R, c["cols"], c["x"])
    elif c["op"] == "expert_combine":
        X = TORCH[c["x"]]
        s["rows"] = _rows(ids, E)
        s["Y"] = r.normal(R, c["cols"]).to(X)
        if c["weights"]:
            s["weights"] = weights
        if c["back"]:
            s["dD"] = r.normal(T, c["cols"]).to(X)
            s["dY"] = _zeros(R, c["cols"], c["x"])
            s["dweights"] = torch.zeros(T, k, device="cuda")
        else:
            if c["res"]:
                s["residual"] = r.normal(T, c["cols"]).to(X)
            s["D"] = _zeros(T, c["cols"], c["x"])
    else:
        N, K = c["N"], c["K"]
        s["offsets"], s["most"] = _offsets(ids, E)
        a, b = r.normal(R, K), r.normal(E, N, K, scale=K ** -0.5)
        if c["op"] == "expert_linear":
            if c["ab"] in QMAX:
                a, s["scale_a"] = _to_8_bits(a, c["ab"])
                b, s["scale_b"] = _to_8_bits(b, c["ab"])
            s["A"], s["B"] = _strided(a.to(TORCH[c["ab"]]), c["pad"]), b.to(TORCH[c["ab"]])
            if c["bias"]:
                s["bias"] = r.normal(E, N, scale=0.2)
            if c["mul"]:
                s["U"] = r.normal(R, N).to(TORCH[c["d"]])
            s["D"] = _zeros(R, N, c["d"], c["pad"])
            if c["z"]:
                s["Z"] = _zeros(R, N, c["d"])
        else:
            X = TORCH[c["ab"]]
            s["A"], s["B"], s["dD"] = a.to(X), b.to(X), r.normal(R, N).to(X)
            if c["act"] != "none":
                s["Z"] = r.normal(R, N).to(X)
                s["dZ"] = _zeros(R, N, c["ab"])
            if c["mul"]:
                s["U"] = r.normal(R, N).to(X)
                s["dU"] = _zeros(R, N, c["ab"])
            s["dA"] = _zeros(R, K, c["ab"])
            if c["db_in"]:
                s["dB_in"] = r.normal(E, N, K, scale=(R / E) ** 0.5)
            s["dB"] = torch.zeros(E, N, K, dtype=TORCH[c["db"]], device="cuda")
            s["dbias"] = torch.zeros(E, N, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
_plans = {}  # a program keeps one plan per problem shape


def _plan(c):
    key = tuple(sorted((k, v) for k, v in c.items() if k != "name"))
    if key not in _plans:
        import beta_epilogue_amd as be
        if c["op"] == "expert_sort":
            _plans[key] = be.ExpertSort(c["T"], c["k"], c["E"], cols=c["cols"], x=c["x"], ids=c["ids"],
                                        scale=c["x"] in QMAX)
        elif c["op"] == "expert_combine" and c["back"]:
            _plans[key] = be.ExpertCombineGrad(c["T"], c["k"], c["cols"], x=c["x"])
        elif c["op"] == "expert_combine":
            _plans[key] = be.ExpertCombine(c["T"], c["k"], c["cols"], x=c["x"], weights=c["weights"],
                                           residual=c["res"])
        elif c["op"] == "expert_linear":
            _plans[key] = be.ExpertLinear(
                c["T"] * c["k"], c["E"], c["N"], c["K"], ab=c["ab"], d=c["d"], act=c["act"],
                bias="f32" if c["bias"] else None, mul=c["mul"], z=c["z"], scale_a=c["ab"] in QMAX,
                scale_b=c["ab"] in QMAX, lda=c["K"] + PAD if c["pad"] else 0, ldd=c["N"] + PAD if c["pad"] else 0)
        elif c["op"] == "expert_linear_grad":
            _plans[key] = be.ExpertLinearGrad(c["T"] * c["k"], c["E"], c["N"], c["K"], ab=c["ab"], act=c["act"],
                                              mul=c["mul"], da=c["ab"], db=c["db"], dbias="f32")
        else:
            _plans[key] = be.AdapterLinear(
                c["M"], c["N"], c["K"], c["r"], c["G"], ab=c["ab"], act=c["act"], bias="f32" if c["bias"] else None,
                residual=c["res"], lda=c["K"] + PAD if c["pad"] else 0, ldd=c["N"] + PAD if c["pad"] else 0)
    return _plans[key]


def _own(s):
    c, op = s["case"], _plan(s["case"])
    if c["op"] == "expert_sort":
        op(s["ids"], s["X"], offsets=s["offsets"], rows=s["rows"], Y=s["Y"], scale=s.get("scale"),
           scale_out=s.get("scale_out"))
        return {k: _values(s[k]) for k in ("offsets", "rows", "Y", "scale_out") if k in s}
    if c["op"] == "expert_combine":
        if c["back"]:
            op(s["dD"], s["Y"], s["rows"], s["weights"], dY=s["dY"], dweights=s["dweights"])
            return {"dY": s["dY"], "dweights": s["dweights"]}
        op(s["Y"], s["rows"], s.get("weights"), residual=s.get("residual"), D=s["D"])
        return {"D": s["D"]}
    if c["op"] == "expert_linear":
        op(s["A"], s["B"], s["offsets"], bias=s.get("bias"), scale_a=s.get("scale_a"), scale_b=s.get("scale_b"),
           U=s.get("U"), D=s["D"], Z=s.get("Z"))
        return {k: s[k] for k in ("D", "Z") if k in s}
    if c["op"] == "expert_linear_grad":
        op(s["dD"], s["A"], s["B"], s["offsets"], Z=s.get("Z"), U=s.get("U"), dB_in=s.get("dB_in"), dZ=s.get("dZ"),
           dU=s.get("dU"), dA=s["dA"], dB=s["dB"], dbias=s["dbias"])
        return {k: s[k] for k in ("dZ", "dU", "dA", "dB", "dbias") if k in s}
    op(s["A"], s["B"], s["ids"], s["down"], s["up"], s["scale"], bias=s.get("bias"), residual=s.get("residual"),
       D=s["D"])
    return {"D": s["D"]}


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


def _groups(s):
    """The rows as a padded batch of groups and back: each group's row numbers
    and which of them it has; each row's group, place in it and whether it has one."""
    off = s["offsets"].to(torch.int64)
    R, E = s["A"].shape[0], off.numel() - 1
    idx = off[:-1, None] + torch.arange(s["most"], device="cuda")
    has = idx < off[1:, None]
    row = torch.arange(R, device="cuda")
    e = torch.searchsorted(off[1:].contiguous(), row, right=True)
    live = e < E
    e = e.clamp(max=E - 1)
    return idx.clamp(max=R - 1), has, e, (row - off[e]).clamp(max=s["most"] - 1), live


def _plain(s):
    c = s["case"]
    if c["op"] == "expert_sort":
        E, flat = c["E"], s["ids"].reshape(-1).to(torch.int64)
        key = torch.where((flat >= 0) & (flat < E), flat, E)
        sorted_key, order = torch.sort(key, stable=True)
        rows = torch.empty_like(flat)
        rows[order] = torch.arange(flat.numel(), device="cuda")
        live = sorted_key < E
        y = torch.where(live[:, None], s["X"].float()[order // c["k"]], 0.0).to(TORCH[c["x"]])
        out = {"offsets": torch.searchsorted(sorted_key, torch.arange(E + 1, device="cuda")).to(torch.int32),
               "rows": torch.where(key < E, rows, -1).to(torch.int32).reshape(s["ids"].shape), "Y": _values(y)}
        if "scale" in s:
            out["scale_out"] = torch.where(live, s["scale"][order // c["k"]], 0.0)
        return out
    if c["op"] == "expert_combine":
        rows, T = s["rows"].to(torch.int64), TORCH[c["x"]]
        live = rows >= 0
        y = torch.where(live[:, :, None], s["Y"].float()[rows.clamp(min=0)], 0.0)
        if c["back"]:
            dd = s["dD"].float()
            # (choices of no expert go to a row behind the last)
            dy = torch.zeros(s["Y"].shape[0] + 1, c["cols"], device="cuda")
            dy[torch.where(live, rows, c["T"] * c["k"])] = s["weights"][:, :, None] * dd[:, None, :]
            return {"dY": dy[:-1].to(T), "dweights": (y * dd[:, None, :]).sum(dim=2)}
        if c["weights"]:
            y = y * s["weights"][:, :, None]
        d = y.sum(dim=1)
        if c["res"]:
            d = d + s["residual"].float()
        return {"D": d.to(T)}
    if c["op"] == "expert_linear":
        T = TORCH[c["d"]]
        idx, _, e, at, live = _groups(s)
        z = torch.bmm(s["A"].float()[idx], s["B"].float().transpose(1, 2).contiguous())
        if "scale_b" in s:
            z = z * s["scale_b"][:, None, :]
        z = z[e, at]
        if "scale_a" in s:
            z = z * s["scale_a"][:, None]
        if c["bias"]:
            z = z + s["bias"][e]
        z = torch.where(live[:, None], z, 0.0)
        d = _act(z, c["act"])
        if c["mul"]:
            d = d * s["U"].float()
        return {"D": d.to(T), "Z": z.to(T)} if c["z"] else {"D": d.to(T)}
    if c["op"] == "expert_linear_grad":
        T = TORCH[c["ab"]]
        idx, has, e, at, live = _groups(s)
        dd = torch.where(live[:, None], s["dD"].float(), 0.0)
        out = {}
        dz = dd
        if c["mul"]:
            out["dU"] = (dd * _act(s["Z"].float(), c["act"])).to(T)
            dz = dz * s["U"].float()
        if c["act"] != "none":
            dz = dz * _act_slope(s["Z"].float(), c["act"])
            out["dZ"] = dz.to(T)
        g = torch.where(has[:, :, None], dz[idx], 0.0)
        db = torch.bmm(g.transpose(1, 2).contiguous(), s["A"].float()[idx])
        if c["db_in"]:
            db = db + s["dB_in"]
        da = torch.where(live[:, None], torch.bmm(g, s["B"].float())[e, at], 0.0)
        return dict(out, dA=da.to(T), dB=db.to(TORCH[c["db"]]), dbias=g.sum(dim=1))
    M, G, r = c["M"], c["G"], c["r"]
    a = s["A"].float()
    z = torch.mm(a, s["B"].float().t())
    # every adapter's inner products, those of other adapters than a row's own set to 0
    u = torch.mm(a, s["down"].float().reshape(G * r, -1).t()).reshape(M, G, r)
    mine = (s["ids"][:, None] == torch.arange(G, device="cuda")) * s["scale"]
    u = (u * mine[:, :, None]).reshape(M, G * r)
    z = z + torch.mm(u, s["up"].float().transpose(1, 2).reshape(G * r, -1))
    if c["bias"]:
        z = z + s["bias"]
    d = _act(z, c["act"])
    if c["res"]:
        d = d + s["residual"].float()
    return {"D": d.to(TORCH[c["ab"]])}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "adapter_linear":
        M, N, K, r, G, es = c["M"], c["N"], c["K"], c["r"], c["G"], SIZE[c["ab"]]
        # adapters that some row has (of G, and no adapter for one row in G + 1)
        met = G * (1.0 - (1.0 - 1.0 / (G + 1)) ** (min(M, 8) if c["runs"] else M))
        n = es * (M * K + N * K + M * N * (1 + c["res"]) + met * r * (N + K)) + 4 * M + (4 * N if c["bias"] else 0)
        return {"bytes": int(n), "flops": 2 * M * N * K + 2 * M * r * (N + K) * G // (G + 1)}
    T, k, E = c["T"], c["k"], c["E"]
    live = (T - c["empty"]) * k
    if c["op"] == "expert_sort":
        n = T * k * ((8 if c["ids"] == "i64" else 4) + 4) + 4 * (E + 1)
        n += (T - c["empty"] + live) * (c["cols"] * SIZE[c["x"]] + (4 if c["x"] in QMAX else 0))
        return {"bytes": n, "flops": 0}
    if c["op"] == "expert_combine":
        row = c["cols"] * SIZE[c["x"]]
        n = 4 * T * k * (1 + c["weights"] + c["back"])
        if c["back"]:
            return {"bytes": n + row * (T + 2 * live), "flops": 3 * live * c["cols"]}
        return {"bytes": n + row * (live + T * (1 + c["res"])), "flops": 2 * live * c["cols"]}
    N, K, es = c["N"], c["K"], SIZE[c["ab"]]
    # experts that some token has, if all are liked alike
    met = E * (1.0 - (1.0 - k / E) ** (T - c["empty"]))
    if c["op"] == "expert_linear":
        ds = SIZE[c["d"]]
        n = live * K * es + live * N * ds * (1 + c["mul"] + c["z"]) + met * N * (K * es + (4 if c["bias"] else 0))
        n += 4 * (E + 1) + (4 * (live + met * N) if c["ab"] in QMAX else 0)
        return {"bytes": int(n), "flops": 2 * live * N * K}
    act = c["act"] != "none"
    n = es * live * (N * (1 + 2 * act + 2 * c["mul"]) + 2 * K) + es * met * N * K + 4 * E * N
    n += E * N * K * SIZE[c["db"]] * (1 + c["db_in"])
    return {"bytes": int(n), "flops": 4 * live * N * K}


def _act64(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


def _slope64(z, act):
    norm = math.sqrt(2.0 / math.pi)
    if act == "relu":
        return torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2.0 * math.pi)
    if act == "none":
        return torch.ones_like(z)
    u, du = (z, 1.0) if act == "silu" else (2.0 * norm * (z + 0.044715 * z ** 3),
                                            2.0 * norm * (1.0 + 3.0 * 0.044715 * z ** 2))
    p = torch.sigmoid(u)
    return p + z * p * (1.0 - p) * du


def exact(case, seed):
    """The definition in 64 bits, group by group."""
    c, s = case, prepare(case, seed)
    f = {k: v.to(torch.float32).to(torch.float64) for k, v in s.items() if torch.is_tensor(v) and k != "B"}
    if c["op"] == "adapter_linear":
        z = f["A"] @ s["B"].to(torch.float64).T
        if c["bias"]:
            z += f["bias"]
        for g in range(c["G"]):
            own_rows = (s["ids"] == g).nonzero()[:, 0]
            z[own_rows] += f["scale"][g] * ((f["A"][own_rows] @ f["down"][g].T) @ f["up"][g].T)
        d = _act64(z, c["act"])
        return {"D": d + f["residual"] if c["res"] else d}
    if c["op"] == "expert_sort":
        rows = [[-1] * c["k"] for _ in range(c["T"])]
        groups = [[] for _ in range(c["E"])]
        for t, choice in enumerate(s["ids"].tolist()):
            for j, e in enumerate(choice):
                if 0 <= e < c["E"]:
                    groups[e].append((t, j))
        off, tokens = [0], []
        for g in groups:
            for t, j in g:
                rows[t][j] = len(tokens)
                tokens.append(t)
            off.append(len(tokens))
        y, t = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda"), torch.tensor(tokens, device="cuda")
        y[:len(tokens)] = f["X"][t]
        out = {"offsets": torch.tensor(off, dtype=torch.int32), "rows": torch.tensor(rows, dtype=torch.int32), "Y": y}
        if "scale" in s:
            out["scale_out"] = torch.zeros(y.shape[0], dtype=torch.float64, device="cuda")
            out["scale_out"][:len(tokens)] = f["scale"][t]
        return out
    if c["op"] == "expert_combine":
        rows = s["rows"].to(torch.int64)
        d = f["residual"].clone() if c["res"] else torch.zeros(c["T"], c["cols"], dtype=torch.float64, device="cuda")
        dy, dw = torch.zeros_like(f["Y"]), torch.zeros(c["T"], c["k"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            t = (rows[:, j] >= 0).nonzero()[:, 0]
            at = rows[t, j]
            w = f["weights"][t, j][:, None] if c["weights"] else 1.0
            if c["back"]:
                dy[at] = w * f["dD"][t]
                dw[t, j] = torch.einsum("tc,tc->t", f["dD"][t], f["Y"][at])
            else:
                d[t] += w * f["Y"][at]
        return {"dY": dy, "dweights": dw} if c["back"] else {"D": d}
    off = s["offsets"].tolist()
    out = {}
    if c["op"] == "expert_linear":
        z = torch.zeros(s["D"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            at = slice(off[e], off[e + 1])
            z[at] = f["A"][at] @ s["B"][e].to(torch.float64).T
            if "scale_a" in f:
                z[at] *= torch.outer(f["scale_a"][at], f["scale_b"][e])
            if c["bias"]:
                z[at] += f["bias"][e]
        d = _act64(z, c["act"])
        out["D"] = d * f["U"] if c["mul"] else d
        if c["z"]:
            out["Z"] = z
        return out
    n = off[-1]
    dz = f["dD"]
    dz[n:] = 0.0
    if c["mul"]:
        out["dU"] = dz * _act64(f["Z"], c["act"])
        dz = dz * f["U"]
    if c["act"] != "none":
        dz = dz * _slope64(f["Z"], c["act"])
        out["dZ"] = dz
    out["dA"] = torch.zeros_like(f["A"])
    out["dB"] = f["dB_in"].clone() if c["db_in"] else torch.zeros(s["dB"].shape, dtype=torch.float64, device="cuda")
    out["dbias"] = torch.zeros_like(f["dbias"])
    for e in range(c["E"]):
        at = slice(off[e], off[e + 1])
        out["dA"][at] = dz[at] @ s["B"][e].to(torch.float64)
        out["dB"][e] += dz[at].T @ f["A"][at]
        out["dbias"][e] = dz[at].sum(0)
    return out
