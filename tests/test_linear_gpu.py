"""The linear layer and its backward on the GPU against plain 64-bit forms
(tests/linear_ref.py, which derives the bounds): every kernel, types, ragged
and smallest sizes, strides with NaN between the rows, values that must not
leak, refusals of a run, streams and graphs.  Each case prints its name before
the GPU step."""
import sys

import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _draw(g, rows, cols, dtype, scale=1.0):
    v = torch.randn(rows, cols, generator=g, dtype=torch.float32) * scale
    if dtype == torch.int8:
        return (v * 40).round().clamp(-127, 127).to(dtype)
    return v.to(dtype)


def _strided(t, pad):
    """A device copy with `pad` elements of NaN (int8: 99) behind every row."""
    if not pad:
        return t.cuda()
    big = torch.full((t.shape[0], t.shape[1] + pad), 99.0 if t.dtype == torch.int8 else NAN).to(t.dtype)
    if t.dtype == torch.float8_e4m3fn:
        big.view(torch.uint8)[:, :t.shape[1]] = t.view(torch.uint8)
    else:
        big[:, :t.shape[1]] = t
    return big.cuda()[:, :t.shape[1]]


SENTINEL = -80.0  # a value of every type


class Out:
    """An output of given row stride between guard rows and columns."""

    def __init__(self, rows, cols, dtype, ld=0):
        self.rows, self.cols, self.ld = rows, cols, ld or cols
        self.buf = torch.full((rows + 2, self.ld), SENTINEL, dtype=torch.float32).to(dtype).cuda()
        # a 16-byte start: a row before it
        self.t = self.buf[1:rows + 1, :cols]

    def intact(self):
        b = self.buf.float()
        return bool((b[0] == SENTINEL).all()) and bool((b[-1] == SENTINEL).all()) and \
            bool((b[1:-1, self.cols:] == SENTINEL).all())


def run_linear(M, N, K, ab, d, act="none", bias=None, res=False, z=False, scaled=False, pad=0, alpha=1.0, splits=0,
               variant=-1, seed=1, inplace=False):
    g = torch.Generator().manual_seed(seed)
    T, DT = ref.TORCH[ab], ref.TORCH[d]
    A, B = _draw(g, M, K, T), _draw(g, N, K, T, 1.0 if ab in ("e4m3", "i8") else K ** -0.5)
    sa = torch.rand(M, generator=g) + 0.5 if scaled else None
    unit = K ** -0.5 * (1 / 1600.0 if ab == "i8" else 1.0)
    sb = (torch.rand(N, generator=g) + 0.5) * unit if scaled else None
    b = _draw(g, 1, N, ref.TORCH[bias])[0] if bias else None
    R = _draw(g, M, N, DT) if res else None
    op = ge.FusedLinear(M, N, K, ab=ab, d=d, act=act, bias=bias, residual=res, z=z, scale_a=scaled, scale_b=scaled,
                        lda=K + pad if pad else 0, ldb=K + pad if pad else 0, ldd=N + pad if pad else 0,
                        ldr=N + pad if pad and res else 0, ldz=N + pad if pad and z else 0, splits=splits,
                        variant=variant)
    D = Out(M, N, DT, N + pad)
    Z = Out(M, N, DT, N + pad) if z else None
    Rd = _strided(R, pad) if res else None
    if inplace:
        D.t.copy_(Rd)
        Rd = D.t
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    args = dict(bias=cuda(b), scale_a=cuda(sa), scale_b=cuda(sb), residual=Rd, Z=Z.t if z else None, alpha=alpha)
    Ad, Bd = _strided(A, pad), _strided(B, pad)
    _say("case", M, N, K, ab, d, act, "pad", pad, op.plan["name"], "splits", op.plan["splits"], "ws",
         op.plan["workspace_bytes"])
    op(Ad, Bd, D=D.t, **args)
    torch.cuda.synchronize()
    assert D.intact() and (Z is None or Z.intact()), "a guard was overwritten"
    dr, zr, S = ref.linear(A, B, act, b, sa, sb, R, alpha)
    fp8 = ab == "e4m3" and d != "f32" and op.plan["name"] != "linear_rows"  # the fp8 MFMA
    bd, bz = ref.linear_bounds(dr, zr, S, K, ab, DT, fp8, R)
    ref.check("D", D.t, dr, bd)
    if z:
        ref.check("Z", Z.t, zr, bz)
    plan = op.plan
    op.close()
    return plan


ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# --- few rows --------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("ab,d", [("bf16", "bf16"), ("f16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"),
                                  ("i8", "f16")])
def test_few_rows(M, ab, d):
    plan = run_linear(M, 264, 656, ab, d, act="silu", bias="f32", res=True, z=True, scaled=ab in ("e4m3", "i8"),
                      seed=M)
    assert plan["name"] == "linear_rows"


@pytest.mark.parametrize("N,K", [(8, 16), (8, 4112), (16, 64), (24, 1040), (4104, 32), (8200, 528)])
@pytest.mark.parametrize("M", [1, 3, 40])
def test_few_rows_sizes(M, N, K):
    run_linear(M, N, K, "bf16", "bf16", bias="bf16", res=True)
    run_linear(M, N, K, "i8", "f32", scaled=True)


def test_few_rows_smallest():
    run_linear(1, 4, 8, "f16", "f32", bias="f16")
    run_linear(1, 4, 16, "e4m3", "f32")


# --- tiles -----------------------------------------------------------------
def test_every_kernel_ragged():
    names = ge.linear_variant_names()
    for v, name in enumerate(names[:-1]):
        ab = name.split("_")[1]
        for d in ("bf16", "f16", "f32"):
            if ab == "e4m3" and (d == "f32") != ("f32" in name):  # a kernel of its own for fp32
                continue
            run_linear(333, 328, 144 + 16 * v, ab, d, act=ACTS[v % 5], bias="f32", res=True, z=True,
                       scaled=ab in ("e4m3", "i8"), variant=v, seed=v)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
def test_activations(act, d):
    run_linear(100, 136, 264, "f16" if d == "f16" else "bf16", d, act=act, bias="f32", z=True, scaled=True, alpha=2.0)


@pytest.mark.parametrize("M,N,K", [(65, 8, 8), (65, 264, 16), (257, 520, 1032), (1001, 256, 40), (300, 2552, 24),
                                   (65, 16, 8200)])
@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_sizes(M, N, K, ab):
    run_linear(M, N, K, ab, ab, act="gelu", bias=ab, res=True)


@pytest.mark.parametrize("splits", [2, 3, 7])
@pytest.mark.parametrize("ab,d", [("bf16", "bf16"), ("f16", "f32"), ("e4m3", "f16"), ("i8", "bf16"), ("e4m3", "f32")])
def test_split_k(splits, ab, d):
    plan = run_linear(270, 264, 1168, ab, d, act="gelu_tanh", bias="f32", res=True, z=True,
                      scaled=ab in ("e4m3", "i8"), splits=splits)
    assert plan["splits"] > 1 and plan["workspace_bytes"] > 0


@pytest.mark.parametrize("M", [5, 130, 300])
@pytest.mark.parametrize("ab,d", [("bf16", "bf16"), ("f16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"), ("i8", "f16")])
def test_strides(M, ab, d):
    """NaN between the rows of every tensor must not reach an output, and what
    lies between the rows of an output stays."""
    run_linear(M, 264, 272, ab, d, act="relu", bias="f32", res=True, z=True, scaled=ab in ("e4m3", "i8"), pad=32)
    run_linear(M, 264, 272, ab, d, scaled=ab == "i8", pad=16, splits=2)


def test_large_rounds():
    """More tiles than compute units, and a last round in K slices."""
    run_linear(4200, 4200, 64, "bf16", "bf16", bias="f32", act="silu")


@pytest.mark.parametrize("M", [7, 200])
def test_residual_in_place(M):
    run_linear(M, 264, 512, "bf16", "bf16", act="gelu", bias="f32", res=True, inplace=True)
    run_linear(M, 264, 512, "bf16", "bf16", res=True, inplace=True, pad=8, splits=2)


@pytest.mark.parametrize("M", [4, 100])
@pytest.mark.parametrize("act", ACTS)
def test_special_values(M, act):
    """A NaN or an infinity of one token's input stays in that token's row;
    an infinite sum gives the activation's limit."""
    N, K = 64, 64
    A = torch.ones(M, K, dtype=torch.bfloat16)
    B = torch.ones(N, K, dtype=torch.bfloat16)
    A[1, 3] = NAN
    A[2, 5] = float("inf")
    op = ge.FusedLinear(M, N, K, act=act, z=True)
    D = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    Z = torch.zeros_like(D)
    _say("case", M, act)
    op(A.cuda(), B.cuda(), D=D, Z=Z)
    D, Z = D.cpu().float(), Z.cpu().float()
    assert torch.isnan(D[1]).all() and torch.isnan(Z[1]).all()
    assert (D[2] == float("inf")).all() and (Z[2] == float("inf")).all()
    rest = [i for i in range(M) if i not in (1, 2)]
    assert (D[rest] == K).all() and (Z[rest] == K).all()


def test_zero_rows_and_zero_scales():
    g = torch.Generator().manual_seed(5)
    for M in (9, 90):
        A = _draw(g, M, 128, torch.bfloat16)
        A[0] = 0
        sa = torch.rand(M, generator=g)
        sa[1] = 0
        B, b = _draw(g, 72, 128, torch.bfloat16), torch.randn(72, generator=g)
        D = torch.empty(M, 72, dtype=torch.bfloat16, device="cuda")
        ge.FusedLinear(M, 72, 128, bias="f32", scale_a=True)(A.cuda(), B.cuda(), bias=b.cuda(), scale_a=sa.cuda(), D=D)
        assert torch.equal(D[0].cpu(), b.bfloat16()) and torch.equal(D[1].cpu(), b.bfloat16())


# --- refusals of a run -----------------------------------------------------
def test_run_refusals():
    M, N, K = 8, 16, 32
    op = ge.FusedLinear(M, N, K, residual=True, bias="f32")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    A, B, R, D = (torch.zeros(*s, **bf) for s in ((M, K), (N, K), (M, N), (M, N)))
    b = torch.zeros(N, device="cuda")
    for bad in (dict(A=A.half()), dict(B=B[:8]), dict(bias=b.half()), dict(bias=None), dict(residual=None),
                dict(D=D.t().contiguous()), dict(Z=D.clone()), dict(A=A.cpu()), dict(scale_a=b[:M])):
        kw = dict(A=A, B=B, bias=b, residual=R, D=D) | bad
        with pytest.raises((ValueError, ge.GemmEpiError)):
            op(kw.pop("A"), kw.pop("B"), **kw)
    wide = torch.zeros(M, K + 4, **bf)
    with pytest.raises(ValueError):  # another row stride
        op(wide[:, :K], B, bias=b, residual=R, D=D)
    off = torch.zeros(M * K + 4, **bf)[4:].view(M, K)  # 8 bytes off
    with pytest.raises(ge.GemmEpiError) as e:
        op(off, B, bias=b, residual=R, D=D)
    assert e.value.code == ge.GEMM_EPI_ERR_ALIGNMENT
    square = ge.FusedLinear(16, 16, 16)
    S, T = (torch.zeros(16, 16, **bf) for _ in range(2))
    for a, w, d in ((S, T, S), (S, T, T)):
        with pytest.raises(ge.GemmEpiError) as e:
            square(a, w, D=d)
        assert e.value.code == ge.GEMM_EPI_ERR_INVALID_ARG
    split = ge.FusedLinear(128, 128, 512, splits=2)
    X = torch.zeros(128, 512, **bf)
    need = split.plan["workspace_bytes"]
    assert need > 0
    for n in (0, need - 1):
        with pytest.raises(ge.GemmEpiError):
            split(X, X, D=torch.zeros(128, 128, **bf), workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


# --- streams and graphs ----------------------------------------------------
def _case(M, N, K, ab="bf16", d="bf16", splits=0, seed=3):
    g = torch.Generator().manual_seed(seed)
    A, B = _draw(g, M, K, ref.TORCH[ab]).cuda(), _draw(g, N, K, ref.TORCH[ab], K ** -0.5).cuda()
    return ge.FusedLinear(M, N, K, ab=ab, d=d, act="gelu", splits=splits), A, B


CASES = [(3, 264, 528, "bf16", "bf16", 0), (130, 264, 1056, "bf16", "bf16", 3), (130, 264, 528, "e4m3", "f32", 2),
         (300, 520, 256, "f16", "f16", 0)]


@pytest.mark.parametrize("c", CASES, ids=str)
def test_graph_replays(c):
    """Two graphs of one plan with split-K workspaces, replayed in turn with
    eager work between, equal the eager result bit for bit."""
    M, N, K, ab, d, splits = c
    _say("case", c)
    op, A, B = _case(*c)
    new = lambda: torch.empty(M, N, dtype=ref.TORCH[d], device="cuda")  # noqa: E731
    want = op(A, B, D=new())
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        out, gr = new(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            op(A, B, D=out)
        graphs.append((gr, out))
    for rep in range(3):
        for gr, out in graphs:
            out.zero_()
            torch.cuda.synchronize()
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), rep
        assert torch.equal(op(A, B, D=new()), want)


def test_two_streams_at_once():
    """Calls of one plan on two streams, each with its own workspace."""
    op, A, B = _case(130, 264, 4096, splits=4)
    outs = [torch.empty(130, 264, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    want = op(A, B, D=torch.empty_like(outs[0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        op(A, B, D=o, stream=streams[i % 2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    raw = torch.empty_like(want)
    op(A, B, D=raw, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw, want)


# --- backward --------------------------------------------------------------
def run_grad(M, N, K, ab="bf16", act="none", da=None, db=None, dbias=None, db_in=False, seed=1, alias=None, tile=0, splits=0):
    g = torch.Generator().manual_seed(seed)
    T = ref.TORCH[ab]
    dD, Z = _draw(g, M, N, T), (_draw(g, M, N, T, 1.5) if act != "none" else None)
    A, B = _draw(g, M, K, T), _draw(g, N, K, T, K ** -0.5)
    C = _draw(g, N, K, ref.TORCH[db]) if db_in else None
    op = ge.FusedLinearGrad(M, N, K, ab=ab, act=act, da=da, db=db, dbias=dbias, tile=tile, splits=splits)
    new = lambda r, c, t: Out(r, c, ref.TORCH[t]) if t else None  # noqa: E731
    dA, dB, dZ = new(M, K, da), new(N, K, db), new(M, N, ab if act != "none" else None)
    db1 = new(1, N, dbias)
    dDd, Zd = dD.cuda(), Z.cuda() if Z is not None else None
    t = lambda o: None if o is None else o.t  # noqa: E731
    dzt = t(dZ) if alias is None else {"dD": dDd, "Z": Zd}[alias]
    Cd = C.cuda() if db_in else None
    if db_in and alias == "dD":  # the weight's gradient added up in place
        dB.t.copy_(Cd)
        Cd = dB.t
    _say("case", M, N, K, ab, act, da, db, dbias, db_in, "tile", tile, "splits", splits, "ws", op.workspace_bytes)
    op(dDd, A.cuda() if db else None, B.cuda() if da else None, Z=Zd, dB_in=Cd, dZ=dzt, dA=t(dA), dB=t(dB),
       dbias=db1.t[0] if db1 else None)
    torch.cuda.synchronize()
    for o in (dA, dB, dZ, db1):
        assert o is None or o.intact()
    exact = ref.f64(dD)
    err = torch.zeros_like(exact)
    if act != "none":
        z = ref.f64(Z)
        err = exact.abs() * (1 + z.abs()) * 2.0 ** -20
        exact = exact * ref.act_slope(z, act)
        ref.check("dZ", dzt, exact, err + ref.half_step(exact.abs() + err, T))
        stored = ref.f64(dzt)
    else:
        stored = exact
    a, b = ref.f64(A), ref.f64(B)
    if da:
        want, S = stored @ b, stored.abs() @ b.abs()
        ref.check("dA", dA.t, want, (N + 4) * ref.U * S + ref.half_step(want.abs() + N * ref.U * S, ref.TORCH[da]))
    if db:
        want, S = stored.T @ a, stored.abs().T @ a.abs()
        if db_in:
            want, S = want + ref.f64(C), S + ref.f64(C).abs()
        ref.check("dB", dB.t, want, (M + 4) * ref.U * S + ref.half_step(want.abs() + M * ref.U * S, ref.TORCH[db]))
    if dbias:
        want = exact.sum(0)
        e = err.sum(0) + (M + 4) * ref.U * (exact.abs() + err).sum(0)
        ref.check("dbias", db1.t[0], want, e + ref.half_step(want.abs() + e, ref.TORCH[dbias]))
    op.close()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_grad(ab, act):
    run_grad(333, 264, 136, ab, act, da=ab, db=ab, dbias="f32")


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (2, 264, 40), (63, 16, 520), (65, 520, 16), (129, 256, 256), (700, 8, 264),
                                   (515, 1032, 72)])
def test_grad_sizes(M, N, K):
    run_grad(M, N, K, "bf16", "silu", da="bf16", db="f32", dbias="bf16")
    run_grad(M, N, K, "f16", "none", da="f32", db="f32", dbias="f32", db_in=True)


@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_grad_tiles(ab, tile, splits):
    """Each tile, whole and in K slices, more tiles than fit at once."""
    run_grad(333, 328, 456, ab, "gelu", da=ab, db="f32", dbias="f32", db_in=True, tile=tile, splits=splits)
    run_grad(40, 1288, 2312, ab, "none", da="f32", db=ab, dbias="f32", tile=tile, splits=splits)


def test_grad_parts():
    run_grad(100, 64, 48, "bf16", "gelu", dbias="f16")
    run_grad(100, 64, 48, "bf16", "gelu", da="f32")
    run_grad(100, 64, 48, "bf16", "none", db="bf16", db_in=True)
    run_grad(100, 64, 48, "f16", "none", dbias="f32")


def test_grad_in_place():
    run_grad(200, 72, 64, "bf16", "gelu_tanh", da="bf16", db="f32", dbias="f32", db_in=True, alias="dD")
    run_grad(200, 72, 64, "f16", "gelu", da="f16", db="f16", dbias="f32", alias="Z")


def test_grad_long_contraction_splits():
    run_grad(4097, 64, 72, "bf16", "relu", da="bf16", db="f32", dbias="f32")


@pytest.mark.parametrize("act", ACTS)
def test_grad_against_differences(act):
    """Central differences of the 64-bit forward f = sum(dD * act(A B^T + b))
    along random directions.  The gradients' own rounding (bf16 dZ, fp32 sums)
    is at most 2^-8 of sum |g| |direction| with |g| <= |dZ| |operand| summed;
    the differences add h^2 (h = 1e-4) and 1e-16 / h, below 1e-7 of it."""
    M, N, K = 40, 48, 56
    g = torch.Generator().manual_seed(11)
    A, B = _draw(g, M, K, torch.bfloat16), _draw(g, N, K, torch.bfloat16, K ** -0.5)
    b = torch.randn(N, generator=g)
    _, z, _ = ref.linear(A, B, "none", b)
    Z = z.to(torch.bfloat16)
    dD = _draw(g, M, N, torch.bfloat16)
    # the forward at which Z is exact: the bias of every element takes what
    # rounding took from z
    shift = ref.f64(Z) - z
    if act == "relu":  # no difference may step over the kink
        dD = torch.where(ref.f64(Z).abs() < 0.02, torch.zeros_like(dD), dD)
    op = ge.FusedLinearGrad(M, N, K, act=act, da="f32", db="f32", dbias="f32")
    dev = dict(device="cuda")
    dA, dB, db = torch.empty(M, K, **dev), torch.empty(N, K, **dev), torch.empty(N, **dev)
    kw = {} if act == "none" else dict(Z=Z.cuda(), dZ=torch.empty(M, N, dtype=torch.bfloat16, **dev))
    _say("case", act)
    op(dD.cuda(), A.cuda(), B.cuda(), dA=dA, dB=dB, dbias=db, **kw)
    a, w, bb = ref.f64(A), ref.f64(B), b.double()

    def f(a, w, bb):
        return (ref.f64(dD) * ref.act(a @ w.T + bb + shift, act)).sum()

    dz = (ref.f64(dD) * ref.act_slope(ref.f64(Z), act)).abs()
    h = 1e-4
    for grad, at, size in ((dA, 0, dz @ w.abs()), (dB, 1, dz.T @ a.abs()), (db, 2, dz.sum(0))):
        u = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        plus, minus = [a, w, bb], [a, w, bb]
        plus[at], minus[at] = plus[at] + h * u, minus[at] - h * u
        diff = float(f(*plus) - f(*minus)) / (2 * h)
        got = float((ref.f64(grad) * u).sum())
        assert abs(got - diff) <= 2.0 ** -8 * float((size * u.abs()).sum()), (act, at, got, diff)


def test_grad_refusals():
    op = ge.FusedLinearGrad(16, 16, 16, act="relu", da="bf16", db="bf16", dbias="f32")
    t = lambda: torch.zeros(16, 16, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    good = dict(dD=t(), A=t(), B=t(), Z=t(), dZ=t(), dA=t(), dB=t(), dbias=torch.zeros(16, device="cuda"))
    assert op(**good) is None
    for bad in (dict(Z=None), dict(dZ=None), dict(A=None), dict(B=None), dict(dA=None), dict(dbias=None),
                dict(dB=good["A"]), dict(dA=good["dD"]), dict(dB=good["dA"]), dict(dD=None),
                dict(dZ=good["A"]), dict(dD=good["dD"].half())):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            op(**(good | bad))
    torch.cuda.synchronize()


@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_grad_infinite_z(act, ab):
    """The slope of an infinite pre-activation (an fp16 overflow) is its limit,
    1 or 0, and a NaN stays in its place."""
    T = ref.TORCH[ab]
    Z = torch.zeros(4, 64, dtype=T)
    Z[0], Z[1], Z[2, 3] = float("inf"), float("-inf"), float("nan")
    dD = torch.full((4, 64), 2.0, dtype=T, device="cuda")
    dZ, db = torch.empty_like(dD), torch.empty(64, device="cuda")
    _say("case", act, ab)
    ge.FusedLinearGrad(4, 64, 64, ab=ab, act=act, dbias="f32")(dD, Z=Z.cuda(), dZ=dZ, dbias=db)
    torch.cuda.synchronize()
    assert (dZ[0] == 2).all() and (dZ[1] == 0).all()
    nan = torch.isnan(dZ[2]).cpu()
    assert nan.sum() <= 1 and bool(nan[3]) == (act != "relu") and torch.isfinite(dZ[3]).all()


def test_grad_graph():
    M, N, K = 260, 264, 520
    g = torch.Generator().manual_seed(4)
    t = lambda r, c: _draw(g, r, c, torch.bfloat16).cuda()  # noqa: E731
    dD, A, B, Z = t(M, N), t(M, K), t(N, K), t(M, N)
    op = ge.FusedLinearGrad(M, N, K, act="gelu", da="bf16", db="f32", dbias="f32")

    def new():
        return dict(dZ=torch.empty_like(dD), dA=torch.empty_like(A), dB=torch.empty(N, K, device="cuda"),
                    dbias=torch.empty(N, device="cuda"))

    want = new()
    op(dD, A, B, Z=Z, **want)
    torch.cuda.synchronize()
    out, graph = new(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(dD, A, B, Z=Z, **out)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), k
        again = new()
        op(dD, A, B, Z=Z, **again)
        assert all(torch.equal(again[k], want[k]) for k in want)


# --- tensors of more than 4 GiB --------------------------------------------
REP = 2100  # of 256 rows; 537600 rows of 8 KiB are 4.4 GB


def _repeats(big, base):
    """Whether `big` is `base` REP times over."""
    n = base.shape[0]
    return all((big[i * n:(i + 1) * n] == base).all() for i in (0, 1, REP // 2 - 1, REP // 2, REP - 2, REP - 1)) and \
        bool((big.view(REP, n, -1) == base).all())


@pytest.mark.parametrize("N,K", [(64, 4096), (4096, 64)])
def test_offsets_beyond_32_bits(N, K):
    """A of 4.4 GB, or D, Z and the residual of 4.4 GB each: every 256 rows
    give what they give alone, bit for bit."""
    variant = ge.linear_variant_names().index("linear_bf16_256x256")
    g = torch.Generator().manual_seed(N)
    A, B, R = (_draw(g, r, c, torch.bfloat16).cuda() for r, c in ((256, K), (N, K), (256, N)))
    out = []
    for rep in (1, REP):
        a, r = A.repeat(rep, 1), R.repeat(rep, 1)
        D, Z = torch.zeros_like(r), torch.zeros_like(r)
        _say("case", rep, N, K)
        ge.FusedLinear(256 * rep, N, K, act="silu", residual=True, z=True, splits=1, variant=variant)(
            a, B, D=D, Z=Z, residual=r)
        out.append((D, Z))
    assert _repeats(out[1][0], out[0][0]) and _repeats(out[1][1], out[0][1])


def test_rows_offsets_beyond_32_bits():
    """One token and a weight of 4.4 GB."""
    g = torch.Generator().manual_seed(8)
    A, B = (_draw(g, r, 4096, torch.bfloat16).cuda() for r in (1, 256))
    want, D = (torch.zeros(1, n, dtype=torch.bfloat16, device="cuda") for n in (256, 256 * REP))
    names = ge.linear_variant_names()
    ge.FusedLinear(1, 256, 4096, variant=names.index("linear_rows"))(A, B, D=want)
    _say("case", 1, 256 * REP, 4096)
    ge.FusedLinear(1, 256 * REP, 4096)(A, B.repeat(REP, 1), D=D)
    assert (D.view(REP, 256) == want).all()


def test_grad_offsets_beyond_32_bits():
    """dD, Z and dZ of 4.4 GB each."""
    g = torch.Generator().manual_seed(9)
    N, K = 4096, 64
    dD, Z, B = torch.ones(256, N, dtype=torch.bfloat16).cuda(), _draw(g, 256, N, torch.bfloat16).cuda(), \
        _draw(g, N, K, torch.bfloat16).cuda()
    out = []
    for rep in (1, REP):
        d, z = dD.repeat(rep, 1), Z.repeat(rep, 1)
        dZ, dA, db = torch.zeros_like(d), torch.zeros(256 * rep, K, dtype=torch.bfloat16, device="cuda"), \
            torch.zeros(N, device="cuda")
        _say("case", rep, N, K)
        ge.FusedLinearGrad(256 * rep, N, K, act="relu", da="bf16", dbias="f32", tile=256, splits=1)(
            d, B=B, Z=z, dZ=dZ, dA=dA, dbias=db)
        out.append((dZ, dA, db))
    assert _repeats(out[1][0], out[0][0]) and _repeats(out[1][1], out[0][1])
    assert (out[1][2] == out[0][2] * REP).all()  # counts below 2^24
