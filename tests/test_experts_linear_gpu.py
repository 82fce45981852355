"""The experts' linear layer and its backward on the GPU against plain 64-bit
forms, expert by expert (tests/linear_ref.py derives the bounds): every kernel,
types, ragged, empty and lopsided experts, strides with NaN between the rows
and in rows behind the last, refusals of a run, streams and graphs, and a whole
mixture of experts forward and backward.  Each case prints its name before the
GPU step."""
import pytest
import torch

import beta_epilogue_amd as ge
import experts_ref as eref
import linear_ref as ref
from test_linear_gpu import ACTS, NAN, Out, _draw, _say, _strided

pytestmark = pytest.mark.gpu

TORCH = ref.TORCH


def sizes(g, R, E, kind):
    """Rows of each expert, R or fewer in all."""
    if kind == "one":
        n = [0] * E
        n[E // 2] = R
    elif kind == "none":
        n = [0] * E
    else:  # uneven, some empty, and (kind "less") fewer rows than the batch holds
        cut = torch.randint(0, R + 1, (E - 1,), generator=g).sort().values.tolist()
        n = [b - a for a, b in zip([0] + cut, cut + [R])]
        if kind == "less":
            n[-1] = n[-1] // 2
    off = [0]
    for v in n:
        off.append(off[-1] + v)
    return off


def _cuda(t):
    return None if t is None else t.cuda()


def run(R, E, N, K, ab, d, act="none", bias=None, mul=False, z=False, scaled=False, pad=0, variant=-1, seed=1,
        kind="uneven", inplace=False):
    g = torch.Generator().manual_seed(seed)
    T, DT = TORCH[ab], TORCH[d]
    off = sizes(g, R, E, kind)
    n = off[-1]
    A = _draw(g, R, K, T)
    B = _draw(g, E * N, K, T, 1.0 if ab in ("e4m3", "i8") else K ** -0.5).view(E, N, K)
    if T.is_floating_point and T != torch.float8_e4m3fn:
        A[n:] = NAN
    sa = torch.rand(R, generator=g) + 0.5 if scaled else None
    unit = K ** -0.5 * (1 / 1600.0 if ab == "i8" else 1.0)
    sb = (torch.rand(E, N, generator=g) + 0.5) * unit if scaled else None
    b = _draw(g, E, N, TORCH[bias]) if bias else None
    U = _draw(g, R, N, DT) if mul else None
    ld = lambda c, on=True: c + pad if pad and on else 0  # noqa: E731
    op = ge.ExpertLinear(R, E, N, K, ab=ab, d=d, act=act, bias=bias, mul=mul, z=z, scale_a=scaled, scale_b=scaled,
                         lda=ld(K), ldd=ld(N), ldu=ld(N, mul), ldz=ld(N, z), variant=variant)
    D = Out(R, N, DT, N + pad)
    Z = Out(R, N, DT, N + pad) if z else None
    Ud = _strided(U, pad) if mul else None
    if inplace:
        D.t.copy_(Ud)
        Ud = D.t
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    _say("case", R, E, N, K, ab, d, act, kind, "mul", mul, "pad", pad, op.plan["name"])
    op(_strided(A, pad), B.cuda(), offsets, D=D.t, bias=_cuda(b), scale_a=_cuda(sa), scale_b=_cuda(sb), U=Ud,
       Z=Z.t if z else None)
    torch.cuda.synchronize()
    assert D.intact() and (Z is None or Z.intact()), "a guard was overwritten"
    if not inplace:
        assert (D.t[n:].float() == -80.0).all(), "rows behind the last were written"
    elif n < R:
        assert torch.equal(D.t[n:].cpu(), U[n:])
    assert not z or (Z.t[n:].float() == -80.0).all()
    plan = op.plan
    fp8 = ab == "e4m3" and d != "f32" and "rows" not in plan["name"]  # the fp8 MFMA
    for e in range(E):
        at = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        dr, zr, S = ref.linear(A[at], B[e], act, b[e] if bias else None, sa[at] if scaled else None,
                               sb[e] if scaled else None)
        acc = 1e-3 if fp8 else (2 * ref.U if ab == "i8" else K * ref.U)
        ez = (acc + 4 * ref.U) * S
        ed = 1.13 * ez + zr.abs() * 2.0 ** -21 + ref.U * zr.abs()
        if mul:
            u = ref.f64(U[at])
            dr, ed = dr * u, ed * u.abs() + ref.U * (dr * u).abs()
        ref.check("D of %d" % e, D.t[at], dr, ed + ref.half_step(dr.abs() + ed, DT))
        if z:
            ref.check("Z of %d" % e, Z.t[at], zr, ez + ref.half_step(zr.abs() + ez, DT))
    op.close()
    return plan


NAMES = ge.expert_linear_variant_names()


@pytest.mark.parametrize("variant", range(len(NAMES)), ids=NAMES)
def test_every_kernel(variant):
    """Groups that end inside tiles, experts without rows, one with all."""
    name = NAMES[variant]
    for ab in ("f16", "bf16", "e4m3", "i8"):
        for d in ("bf16", "f16", "f32"):
            if "rows" not in name and (name.split("_")[1] != ab or (ab == "e4m3" and (d == "f32") != ("f32" in name))):
                continue
            q = ab in ("e4m3", "i8")
            run(700, 9, 328, 144 + 16 * variant, ab, d, act=ACTS[variant % 5], bias="f32", mul=True, z=True, scaled=q,
                variant=variant, seed=variant)
            run(300, 3, 136, 272, ab, d, scaled=q, variant=variant, kind="one", pad=16)
            run(90, 33, 72, 80, ab, d, scaled=q, variant=variant, kind="less", act="silu")


@pytest.mark.parametrize("rows,cols", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("variant", range(len(NAMES)), ids=NAMES)
def test_scales(variant, rows, cols):
    """Row scales and each expert's column scales, alone and together, in every kernel
    and type, with uneven and empty experts (bounds as in ``run``)."""
    name, R, E, N, K = NAMES[variant], 333, 6, 136, 208
    for ab, d in (("bf16", "bf16"), ("f16", "f16"), ("e4m3", "f16"), ("e4m3", "f32"), ("i8", "bf16")):
        wide = ab == "e4m3" and d == "f32"
        if "rows" not in name and (name.split("_")[1] != ab or wide != ("f32" in name)):
            continue
        g = torch.Generator().manual_seed(variant)
        off = [0, 0, 70, 201, 201, 330, 330]
        unit = K ** -0.5 * (1 / 1600.0 if ab == "i8" else 1.0)
        A, B = _draw(g, R, K, TORCH[ab]), _draw(g, E * N, K, TORCH[ab]).view(E, N, K)
        sa = (torch.rand(R, generator=g) + 0.5) * unit if rows else None
        sb = (torch.rand(E, N, generator=g) + 0.5) * (1.0 if rows else unit) if cols else None
        op = ge.ExpertLinear(R, E, N, K, ab=ab, d=d, scale_a=rows, scale_b=cols, variant=variant)
        D = Out(R, N, TORCH[d])
        _say("case scales", name, ab, d, rows, cols)
        op(A.cuda(), B.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"), D=D.t, scale_a=_cuda(sa), scale_b=_cuda(sb))
        torch.cuda.synchronize()
        assert D.intact() and (D.t[off[-1]:].float() == -80.0).all()
        fp8 = ab == "e4m3" and not wide and "rows" not in name
        acc = 1e-3 if fp8 else (2 * ref.U if ab == "i8" else K * ref.U)
        for e in range(E):
            at = slice(off[e], off[e + 1])
            if off[e] < off[e + 1]:
                dr, _, S = ref.linear(A[at], B[e], "none", None, sa[at] if rows else None, sb[e] if cols else None)
                ed = (acc + 4 * ref.U) * S
                ref.check("D of %d" % e, D.t[at], dr, ed + ref.half_step(dr.abs() + ed, TORCH[d]))


@pytest.mark.parametrize("R,E", [(1, 1), (1, 64), (8, 64), (15, 4), (64, 3), (65, 65), (128, 1024), (500, 100), (3000, 7)])
@pytest.mark.parametrize("ab,d", [("bf16", "bf16"), ("f16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"), ("i8", "f16")])
def test_rows_and_experts(R, E, ab, d):
    q = ab in ("e4m3", "i8")
    run(R, E, 40, 208, ab, d, act="gelu", bias="f32", mul=True, scaled=q, seed=R)
    run(R, E, 16, 16, ab, d, scaled=q, seed=R, kind="less")


@pytest.mark.parametrize("kind", ["one", "none", "less"])
@pytest.mark.parametrize("R", [6, 400])
def test_lopsided(kind, R):
    for v in range(-1, len(NAMES)):
        if v >= 0 and "rows" not in NAMES[v] and "bf16" not in NAMES[v]:
            continue
        run(R, 6, 72, 136, "bf16", "bf16", act="silu", mul=True, z=True, variant=v, kind=kind)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
def test_activations(act, d):
    run(150, 4, 136, 264, "f16" if d == "f16" else "bf16", d, act=act, bias="f32", mul=True, z=True)


@pytest.mark.parametrize("R,E,N,K", [(65, 2, 8, 8), (300, 4, 264, 16), (600, 2, 520, 1032), (4100, 3, 520, 64),
                                     (200, 5, 16, 8200)])
def test_sizes(R, E, N, K):
    run(R, E, N, K, "bf16", "bf16", act="gelu", bias="bf16", mul=True)
    run(R, E, N, K, "f16", "f16", bias="f16")


@pytest.mark.parametrize("R", [9, 260])
def test_factor_in_place(R):
    run(R, 4, 264, 512, "bf16", "bf16", act="silu", mul=True, inplace=True, kind="less")
    run(R, 4, 264, 512, "bf16", "bf16", act="silu", mul=True, inplace=True, pad=8, kind="less")


def test_the_plan_follows_the_rows():
    assert "rows" in ge.ExpertLinear(8, 64, 1024, 2048).plan["name"]
    assert "256" in ge.ExpertLinear(32768, 8, 4096, 4096).plan["name"]


@pytest.mark.parametrize("K", [128, 1040])
def test_sums_of_e4m3(K):
    """Large products that cancel among small ones: fp32's precision where e4m3 is widened
    (the few-row kernels, fp32 outputs), 0.001 of the sum of |a||b| where the fp8 matrix
    instructions sum."""
    R, N, T8 = 200, 136, torch.float8_e4m3fn
    g = torch.Generator().manual_seed(K)
    A, B = torch.rand(R, K, generator=g) + 0.5, torch.ones(1, N, K)
    for d in ("f16", "f32"):
        for size in (64.0, 2048.0, 8192.0, 65536.0):
            A[:, 3], A[:, K // 2 + 5], B[:, :, 3], B[:, :, K // 2 + 5] = size / 256, -size / 256, 256.0, 256.0
            a, b = A.to(T8), B.to(T8)
            for v, name in enumerate(NAMES):
                if "rows" not in name and ("e4m3" not in name or (d == "f32") != ("f32" in name)):
                    continue
                D = torch.empty(R, N, dtype=TORCH[d], device="cuda")
                _say("case cancel", name, d, size)
                ge.ExpertLinear(R, 1, N, K, ab="e4m3", d=d, variant=v)(
                    a.cuda(), b.cuda(), torch.tensor([0, R], dtype=torch.int32, device="cuda"), D=D)
                dr, _, S = ref.linear(a, b[0])
                e = (K * ref.U if "rows" in name or d == "f32" else 1e-3) * S
                ref.check("D", D, dr, e + ref.half_step(dr.abs() + e, TORCH[d]))


def test_special_values():
    """A NaN or an infinity of one row stays in it; infinite factors follow the
    formula (0 * infinity is NaN)."""
    for R in (6, 200):
        A = torch.ones(R, 64, dtype=torch.bfloat16)
        B = torch.ones(2, 64, 64, dtype=torch.bfloat16)
        A[1, 3], A[2, 5], A[4] = NAN, float("inf"), 0.0
        U = torch.ones(R, 64, dtype=torch.bfloat16)
        U[3], U[4] = float("inf"), float("inf")
        off = torch.tensor([0, 3, R], dtype=torch.int32, device="cuda")
        D = torch.zeros(R, 64, dtype=torch.bfloat16, device="cuda")
        _say("case special", R)
        ge.ExpertLinear(R, 2, 64, 64, act="relu", mul=True)(A.cuda(), B.cuda(), off, U=U.cuda(), D=D)
        D = D.cpu().float()
        assert torch.isnan(D[1]).all() and (D[2] == float("inf")).all() and (D[3] == float("inf")).all()
        assert torch.isnan(D[4]).all() and (D[0] == 64).all() and (D[5:] == 64).all()


def test_offsets_outside_the_batch():
    """Offsets that do not ascend, or lie outside the rows: nothing outside the
    tensors is touched, and experts whose rows are sound get theirs."""
    R, E, N, K = 40, 4, 64, 64
    A, B = torch.ones(R, K, dtype=torch.bfloat16, device="cuda"), torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda")
    for off in ([-5, 10, 20, 1000, 2000], [0, 30, 10, 1 << 30, -(1 << 31)]):
        for v, name in enumerate(NAMES):
            if "rows" in name or "bf16" in name:
                D = Out(R, N, torch.bfloat16)
                _say("case offsets", off, name)
                ge.ExpertLinear(R, E, N, K, variant=v)(A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), D=D.t)
                torch.cuda.synchronize()
                assert D.intact() and (D.t[:10] == K).all()


# --- backward --------------------------------------------------------------
def run_grad(R, E, N, K, ab="bf16", act="none", mul=False, da=None, db=None, dbias=None, db_in=False, seed=1, tile=0,
             kind="uneven", alias=None):
    g = torch.Generator().manual_seed(seed)
    T = TORCH[ab]
    off = sizes(g, R, E, kind)
    n = off[-1]
    has_z = act != "none" or mul
    dD, A = _draw(g, R, N, T), _draw(g, R, K, T)
    Z, U = (_draw(g, R, N, T, 1.5) if has_z else None), (_draw(g, R, N, T) if mul else None)
    B = _draw(g, E * N, K, T, K ** -0.5).view(E, N, K)
    C = _draw(g, E * N, K, TORCH[db]).view(E, N, K) if db_in else None
    for t in (dD, A, Z, U):
        if t is not None:
            t[n:] = NAN
    op = ge.ExpertLinearGrad(R, E, N, K, ab=ab, act=act, mul=mul, da=da, db=db, dbias=dbias, tile=tile)
    new = lambda r, c, t: Out(r, c, TORCH[t]) if t else None  # noqa: E731
    dA, dB, dZ, dU, db1 = (new(R, K, da), new(E * N, K, db), new(R, N, ab if has_z else None),
                           new(R, N, ab if mul else None), new(E, N, dbias))
    dDd, Zd, Ud, Cd = dD.cuda(), _cuda(Z), _cuda(U), _cuda(C)
    t = lambda o: None if o is None else o.t  # noqa: E731
    dzt, dut, dbt = t(dZ), t(dU), dB.t.view(E, N, K) if dB else None
    if alias:
        dzt, dut = {"dD": dDd, "Z": Zd}[alias], Ud
        if db_in:
            dbt.copy_(Cd)
            Cd = dbt
    _say("case grad", R, E, N, K, ab, act, mul, da, db, dbias, db_in, kind, "tile", tile, "ws", op.workspace_bytes)
    op(dDd, A.cuda() if db else None, B.cuda() if da else None, torch.tensor(off, dtype=torch.int32, device="cuda"),
       Z=Zd, U=Ud, dB_in=Cd, dZ=dzt, dU=dut, dA=t(dA), dB=dbt, dbias=t(db1))
    torch.cuda.synchronize()
    for o in (dA, dB, dZ, dU, db1):
        assert o is None or o.intact()
    for o in (dA, dZ, dU):
        assert o is None or alias or (o.t[n:].float() == -80.0).all(), "rows behind the last were written"
    exact = ref.f64(dD)[:n]
    err = torch.zeros_like(exact)
    if has_z:
        z = ref.f64(Z)[:n]
        if mul:
            du = exact * ref.act(z, act)
            e = exact.abs() * z.abs() * 2.0 ** -20
            ref.check("dU", dut[:n], du, e + ref.half_step(du.abs() + e, T))
            exact = exact * ref.f64(U)[:n]
        err = exact.abs() * (1 + z.abs()) * 2.0 ** -20
        exact = exact * ref.act_slope(z, act)
        ref.check("dZ", dzt[:n], exact, err + ref.half_step(exact.abs() + err, T))
        stored = ref.f64(dzt)[:n]
    else:
        stored = exact
    a = ref.f64(A)
    for e in range(E):
        at = slice(off[e], off[e + 1])
        m, s, b = off[e + 1] - off[e], stored[at], ref.f64(B[e])
        if da and m:
            want, S = s @ b, s.abs() @ b.abs()
            ref.check("dA of %d" % e, dA.t[at], want,
                      (N + 4) * ref.U * S + ref.half_step(want.abs() + N * ref.U * S, TORCH[da]))
        if db:
            want, S = s.T @ a[at], s.abs().T @ a[at].abs()
            if db_in:
                want, S = want + ref.f64(C[e]), S + ref.f64(C[e]).abs()
            ref.check("dB of %d" % e, dbt[e], want,
                      (m + 4) * ref.U * S + ref.half_step(want.abs() + m * ref.U * S, TORCH[db]))
        if dbias:
            want = exact[at].sum(0)
            er = err[at].sum(0) + (m + 4) * ref.U * (exact[at].abs() + err[at]).sum(0)
            ref.check("dbias of %d" % e, db1.t[e], want, er + ref.half_step(want.abs() + er, TORCH[dbias]))
    op.close()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_grad(ab, act):
    run_grad(333, 5, 264, 136, ab, act, da=ab, db=ab, dbias="f32")
    run_grad(333, 5, 264, 136, ab, act, mul=True, da=ab, db="f32", dbias="f32", kind="less")


@pytest.mark.parametrize("R,E,N,K", [(1, 1, 8, 8), (1, 9, 8, 8), (2, 2, 264, 40), (63, 4, 16, 520), (65, 70, 520, 16),
                                     (300, 2, 256, 256), (700, 3, 8, 264), (515, 1024, 24, 72), (2100, 2, 72, 72)])
def test_grad_sizes(R, E, N, K):
    run_grad(R, E, N, K, "bf16", "silu", mul=True, da="bf16", db="f32", dbias="bf16")
    run_grad(R, E, N, K, "f16", "none", da="f32", db="f32", dbias="f32", db_in=True)


@pytest.mark.parametrize("kind", ["uneven", "one", "none", "less"])
@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("ab", ["bf16", "f16"])
def test_grad_tiles(ab, tile, kind):
    """Each tile, experts that end inside tiles and K tiles, without rows, and one
    with all."""
    run_grad(700, 4, 328, 456, ab, "gelu", da=ab, db="f32", dbias="f32", db_in=True, tile=tile, kind=kind)
    run_grad(150, 7, 72, 520, ab, "none", da="f32", db=ab, dbias="f16", tile=tile, kind=kind)


@pytest.mark.parametrize("act,mul", [("none", False), ("gelu", True)])
def test_grad_in_ranges_of_rows(act, mul):
    """A batch in several calls, with offsets less each range's first row: rows of other
    ranges are neither read nor written, and dB goes on from the range before."""
    R, E, N, K, T = 700, 6, 264, 136, torch.bfloat16
    g = torch.Generator().manual_seed(11)
    off = [0, 0, 130, 395, 395, 640, 690]
    dD, A, Z, U = (_draw(g, R, n, T).cuda() for n in (N, K, N, N))
    B = _draw(g, E * N, K, T, K ** -0.5).view(E, N, K).cuda()
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    has_z = act != "none"
    dA, dZ, dU = Out(R, K, T), Out(R, N, T), Out(R, N, T)
    dB, dbias = torch.zeros(E, N, K, device="cuda"), torch.zeros(E, N, device="cuda")
    for i, (lo, hi) in enumerate(((0, 200), (200, 400), (400, R))):
        op = ge.ExpertLinearGrad(hi - lo, E, N, K, act=act, mul=mul, da="bf16", db="f32", dbias="f32")
        part, more = torch.empty_like(dbias), {}
        if has_z:
            more = dict(Z=Z[lo:hi], U=U[lo:hi], dZ=dZ.t[lo:hi], dU=dU.t[lo:hi])
        _say("case ranges", act, lo, hi)
        op(dD[lo:hi], A[lo:hi], B, offsets - lo, dA=dA.t[lo:hi], dB=dB, dB_in=dB if i else None, dbias=part, **more)
        dbias += part
    torch.cuda.synchronize()
    assert dA.intact() and dZ.intact() and dU.intact() and (dA.t[off[-1]:].float() == -80.0).all()
    dz = ref.f64(dZ.t if has_z else dD)
    for e in range(E):
        at, m = slice(off[e], off[e + 1]), off[e + 1] - off[e]
        s, a, b = dz[at], ref.f64(A)[at], ref.f64(B)[e]
        want, S = s @ b, s.abs() @ b.abs()
        ref.check("dA of %d" % e, dA.t[at], want, (N + 4) * ref.U * S + ref.half_step(want.abs() + N * ref.U * S, T))
        want, S = s.T @ a, s.abs().T @ a.abs()
        ref.check("dB of %d" % e, dB[e], want, (m + 8) * ref.U * S + ref.half_step(want.abs() + m * ref.U * S, torch.float32))
        # (dbias adds up dZ before its rounding)
        half = ref.half_step(s, T).sum(0) if has_z else 0.0
        ref.check("dbias of %d" % e, dbias[e], s.sum(0), 1.01 * half + (m + 8) * ref.U * s.abs().sum(0) + 1e-30)


def test_grad_more_tiles_than_fit():
    run_grad(2500, 6, 1032, 520, "bf16", "relu", da="bf16", db="bf16", dbias="f32", tile=64)
    run_grad(2500, 6, 1032, 520, "bf16", "relu", da="bf16", db="bf16", tile=128)


@pytest.mark.parametrize("kind", ["uneven", "one", "none", "less"])
@pytest.mark.parametrize("da,db", [("bf16", None), (None, "f32"), ("bf16", "f32")])
def test_grad_bias_of_many_rows(da, db, kind):
    """Without an activation and dB, of more rows than one workgroup adds up in the time
    of a product: any of them may be one expert's, so chunks of them are added up apart
    and joined from the workspace."""
    R, E, N, K = 17000, 5, 328, 72
    run_grad(R, E, N, K, da=da, db=db, dbias="f32", kind=kind)
    need = lambda R, **kw: ge.ExpertLinearGrad(R, E, N, K, da=da, db=db, **kw).workspace_bytes  # noqa: E731
    assert need(R, dbias="f32") >= (0 if db else R // 1024 * N * 4)
    assert need(16384, dbias="f32") == 0 and need(R) == 0


def test_grad_bias_of_many_rows_in_graphs():
    """Two graphs replayed in turn with eager calls between, bit for bit as alone."""
    R, E, N, K = 17000, 5, 72, 72
    g, T = torch.Generator().manual_seed(3), torch.bfloat16
    dD, B = _draw(g, R, N, T).cuda(), _draw(g, E * N, K, T).view(E, N, K).cuda()
    off = torch.tensor(sizes(g, R, E, "uneven"), dtype=torch.int32, device="cuda")
    op = ge.ExpertLinearGrad(R, E, N, K, da="bf16", dbias="f32")
    new = lambda: (torch.zeros(R, K, dtype=T, device="cuda"), torch.zeros(E, N, device="cuda"))  # noqa: E731
    call = lambda o: op(dD, None, B, off, dA=o[0], dbias=o[1])  # noqa: E731
    _say("case bias in graphs", R, E, N, K)
    want, outs, graphs = new(), [new(), new()], [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    call(want)
    torch.cuda.synchronize()
    for gr, o in zip(graphs, outs):
        with torch.cuda.graph(gr):
            call(o)
    for _ in range(3):
        eager = new()
        for o in outs:
            o[0].zero_(), o[1].zero_()
        for gr in graphs:
            gr.replay()
        call(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o in outs + [eager] for a, b in zip(o, want))


def test_grad_bias_of_many_rows_and_experts():
    run_grad(16385, 1024, 72, 16, "f16", da="f16", dbias="f16")
    run_grad(30000, 2, 1032, 8, "bf16", da="bf16", dbias="bf16", tile=128)
    run_grad(30000, 70, 8, 8, "bf16", db="f32", dbias="f32", tile=256, kind="less")


def test_grad_parts():
    run_grad(100, 3, 64, 48, "bf16", "gelu", dbias="f16")
    run_grad(100, 3, 64, 48, "bf16", "gelu", da="f32")
    run_grad(100, 3, 64, 48, "bf16", "none", db="bf16", db_in=True)
    run_grad(100, 3, 64, 48, "f16", "none", dbias="f32")
    run_grad(100, 3, 64, 48, "f16", "silu", mul=True)
    run_grad(100, 3, 64, 48, "f16", "none", mul=True, da="f16")


@pytest.mark.parametrize("R", [333, 17000])
@pytest.mark.parametrize("act,mul", [("none", False), ("silu", True)])
@pytest.mark.parametrize("tile", [64, 128, 256])
def test_grad_of_one_experts_nans(tile, act, mul, R):
    """NaN and infinities in one expert's first and last rows reach its own gradients,
    and change no bit of the other experts'."""
    E, N, K, T = 4, 72, 136, torch.bfloat16
    g = torch.Generator().manual_seed(R)
    off = [0, 5, R // 2 + 3, R - 9, R]
    mine = slice(off[1], off[2])
    has_z = act != "none"
    clean = dict(dD=_draw(g, R, N, T), A=_draw(g, R, K, T), Z=_draw(g, R, N, T), U=_draw(g, R, N, T))
    B = _draw(g, E * N, K, T, K ** -0.5).view(E, N, K).cuda()
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    for wants in (dict(da="bf16", db="f32", dbias="f32"), dict(da="bf16", dbias="f32"), dict(db="f32", dbias="f32")):
        op = ge.ExpertLinearGrad(R, E, N, K, act=act, mul=mul, tile=tile, **wants)
        got = []
        for dirty in (False, True):
            t = {n: v.clone() for n, v in clean.items()}
            if dirty:
                for i, v in enumerate(t.values()):
                    v[off[1], i::7], v[off[2] - 1, i::5] = NAN, float("inf")
            t = {n: v.cuda() for n, v in t.items()}
            e = lambda *s: torch.zeros(*s, dtype=T, device="cuda")  # noqa: E731
            o = dict(dbias=torch.zeros(E, N, device="cuda"))
            if "da" in wants:
                o["dA"] = e(R, K)
            if "db" in wants:
                o["dB"] = torch.zeros(E, N, K, device="cuda")
            if has_z:
                o |= dict(dZ=e(R, N), dU=e(R, N))
            _say("case NaN of one expert", R, act, tile, wants, dirty)
            op(t["dD"], t["A"] if "db" in wants else None, B if "da" in wants else None, offsets,
               Z=t["Z"] if has_z else None, U=t["U"] if has_z else None, **o)
            torch.cuda.synchronize()
            got.append({n: v.cpu() for n, v in o.items()})
        for n, want in got[0].items():
            v = got[1][n]
            if n in ("dB", "dbias"):
                assert torch.isnan(v[1]).any() and torch.equal(v[[0, 2, 3]], want[[0, 2, 3]]), n
            else:
                assert torch.isnan(v[mine]).any(), n
                assert torch.equal(v[:off[1]], want[:off[1]]) and torch.equal(v[off[2]:], want[off[2]:]), n


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("tile", [64, 128, 256])
def test_grad_of_offsets_outside_the_batch(tile, act):
    """As in the forward: nothing outside the tensors is touched."""
    R, E, N, K = 40, 4, 64, 72
    T = torch.bfloat16
    x = lambda *s: torch.ones(*s, dtype=T, device="cuda")  # noqa: E731
    dD, A, B = x(R, N), x(R, K), x(E, N, K)
    for off in ([-5, 10, 20, 1000, 2000], [0, 30, 10, 1 << 30, -(1 << 31)], [7] + [(1 << 31) - 1, 0] * 2):
        dA, dB, dbias, dZ = Out(R, K, T), Out(E * N, K, T), Out(E, N, T), Out(R, N, T)
        _say("case gradients of offsets", off, tile, act)
        op = ge.ExpertLinearGrad(R, E, N, K, act=act, da="bf16", db="bf16", dbias="bf16", tile=tile)
        z = dict(Z=dD, dZ=dZ.t) if act != "none" else {}
        op(dD, A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), dA=dA.t, dB=dB.t.view(E, N, K), dbias=dbias.t, **z)
        torch.cuda.synchronize()
        assert dA.intact() and dB.intact() and dbias.intact() and dZ.intact()


def test_grad_bias_of_offsets_outside_many_rows():
    R, E, N, K = 17000, 4, 64, 72
    T = torch.bfloat16
    dD, B = torch.ones(R, N, dtype=T, device="cuda"), torch.ones(E, N, K, dtype=T, device="cuda")
    for off in ([-5, 10, 20, 30000, 40000], [0, 30, 10, 1 << 30, -(1 << 31)], [7] + [(1 << 31) - 1, 0] * 2):
        dA, dbias = Out(R, K, T), Out(E, N, T)
        _say("case bias of offsets", off)
        op = ge.ExpertLinearGrad(R, E, N, K, da="bf16", dbias="bf16")
        op(dD, None, B, torch.tensor(off, dtype=torch.int32, device="cuda"), dA=dA.t, dbias=dbias.t)
        torch.cuda.synchronize()
        assert dA.intact() and dbias.intact()


@pytest.mark.parametrize("alias", ["dD", "Z"])
def test_grad_in_place(alias):
    run_grad(200, 3, 72, 64, "bf16", "gelu_tanh", mul=True, da="bf16", db="f32", dbias="f32", db_in=True, alias=alias)


@pytest.mark.parametrize("kind", ["one", "none"])
@pytest.mark.parametrize("db", ["f32", "bf16"])
def test_grad_in_place_without_rows(db, kind):
    run_grad(90, 5, 72, 200, "bf16", "silu", da="bf16", db=db, db_in=True, alias="dD", kind=kind)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_grad_against_differences(act):
    """Central differences of f = sum(dD * act(A B[e]^T + shift) * U) in 64 bits
    along random directions (shift makes the stored Z exact).  The gradients' own
    rounding is at most 2^-8 of the sums of |g||direction|, and the differences
    (h = 1e-4) add less than 1e-7 of them."""
    R, E, N, K = 60, 3, 40, 48
    g = torch.Generator().manual_seed(12)
    off = [0, 25, 25, 60]
    A, B = _draw(g, R, K, torch.bfloat16), _draw(g, E * N, K, torch.bfloat16, K ** -0.5).view(E, N, K)
    U, dD = _draw(g, R, N, torch.bfloat16), _draw(g, R, N, torch.bfloat16)
    group = torch.tensor([e for e in range(E) for _ in range(off[e + 1] - off[e])])
    product = lambda a, w: torch.einsum("rk,rnk->rn", a, w[group])  # noqa: E731
    Z = product(ref.f64(A), ref.f64(B)).to(torch.bfloat16)
    shift = ref.f64(Z) - product(ref.f64(A), ref.f64(B))
    dev = dict(device="cuda")
    dA, dB, dbias = torch.empty(R, K, **dev), torch.empty(E, N, K, **dev), torch.empty(E, N, **dev)
    dZ, dU = (torch.empty(R, N, dtype=torch.bfloat16, **dev) for _ in range(2))
    _say("case differences", act)
    ge.ExpertLinearGrad(R, E, N, K, act=act, mul=True, da="f32", db="f32", dbias="f32")(
        dD.cuda(), A.cuda(), B.cuda(), torch.tensor(off, dtype=torch.int32, **dev), Z=Z.cuda(), U=U.cuda(), dZ=dZ,
        dU=dU, dA=dA, dB=dB, dbias=dbias)
    a, w, u, b = ref.f64(A), ref.f64(B), ref.f64(U), torch.zeros(E, N, dtype=torch.float64)

    def f(a, w, u, b):
        return (ref.f64(dD) * ref.act(product(a, w) + b[group] + shift, act) * u).sum()

    dz = (ref.f64(dD) * u * ref.act_slope(ref.f64(Z), act)).abs()
    onehot = torch.nn.functional.one_hot(group, E).double()
    size = dict(a=torch.einsum("rn,rnk->rk", dz, w.abs()[group]), w=torch.einsum("re,rn,rk->enk", onehot, dz, a.abs()),
                u=(ref.f64(dD) * ref.act(ref.f64(Z), act)).abs(), b=onehot.T @ dz)
    h, x = 1e-4, dict(a=a, w=w, u=u, b=b)
    for name, grad in (("a", dA), ("w", dB), ("u", dU), ("b", dbias)):
        way = torch.randn(x[name].shape, generator=g, dtype=torch.float64)
        ends = [f(**dict(x, **{name: x[name] + s * h * way})) for s in (1, -1)]
        want, got = (ends[0] - ends[1]) / (2 * h), (ref.f64(grad) * way).sum()
        bound = (2.0 ** -8 + 1e-7) * (size[name] * way.abs()).sum()
        assert abs(want - got) <= bound, (name, float(want), float(got), float(bound))


def test_grad_of_infinite_preactivations():
    """The slope of an infinite pre-activation is its limit."""
    dD = torch.full((4, 64), 2.0, dtype=torch.float16, device="cuda")
    Z = torch.zeros(4, 64, dtype=torch.float16)
    Z[0], Z[1] = float("inf"), -float("inf")
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    for act in ACTS[1:]:
        dZ, db = torch.empty_like(dD), torch.empty(2, 64, device="cuda")
        _say("case infinite", act)
        ge.ExpertLinearGrad(4, 2, 64, 64, ab="f16", act=act, dbias="f32")(dD, None, None, off, Z=Z.cuda(), dZ=dZ, dbias=db)
        assert (dZ[0] == 2).all() and (dZ[1] == 0).all() and torch.isfinite(db).all()


# --- the operators together -------------------------------------------------
def _layer(T, k, E, H, F, seed):
    """A gated mixture of experts: norm, sort, two products in, one out, combine;
    then its backward.  Returns a function of an output set, and a maker of them."""
    g = torch.Generator().manual_seed(seed)
    R, b = T * k, dict(dtype=torch.bfloat16, device="cuda")
    x = _draw(g, T, H, torch.bfloat16)
    ids = torch.topk(torch.randn(T, E, generator=g), k, dim=1).indices
    ids[-2:] = -1
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    w1, w2, w3 = (_draw(g, E * n, m, torch.bfloat16, m ** -0.5).view(E, n, m) for n, m in ((F, H), (F, H), (H, F)))
    dout = _draw(g, T, H, torch.bfloat16)
    host = dict(x=x, ids=ids, w=w, w1=w1, w2=w2, w3=w3, dout=dout)
    dev = {n: v.cuda() for n, v in host.items()}
    sort, back = ge.ExpertSort(T, k, E, cols=H), ge.ExpertCombine(T, k, H, residual=True)
    up, gate = ge.ExpertLinear(R, E, F, H), ge.ExpertLinear(R, E, F, H, act="silu", mul=True, z=True)
    down, dback = ge.ExpertLinear(R, E, H, F), ge.ExpertCombineGrad(T, k, H)
    ddown = ge.ExpertLinearGrad(R, E, H, F, da="bf16", db="f32")
    dgate = ge.ExpertLinearGrad(R, E, F, H, act="silu", mul=True, da="bf16", db="f32")
    dup = ge.ExpertLinearGrad(R, E, F, H, da="bf16", db="f32")
    dsort = ge.ExpertCombine(T, k, H, weights=False, residual=True)

    def new():
        e = lambda *s: torch.zeros(*s, **b)  # noqa: E731
        f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(off=i(E + 1), rows=i(T, k), xs=e(R, H), u=e(R, F), z=e(R, F), h=e(R, F), y=e(R, H), out=e(T, H),
                    dy=e(R, H), dw=f(T, k), dh=e(R, F), dw3=f(E, H, F), dz=e(R, F), du=e(R, F), dxs=e(R, H), dw1=f(E, F, H),
                    dxs2=e(R, H), dw2=f(E, F, H), dx1=e(T, H), dx=e(T, H))

    def call(o, stream=None):
        s, d = dict(stream=stream), dev
        sort(d["ids"], d["x"], offsets=o["off"], rows=o["rows"], Y=o["xs"], **s)
        up(o["xs"], d["w2"], o["off"], D=o["u"], **s)
        gate(o["xs"], d["w1"], o["off"], U=o["u"], Z=o["z"], D=o["h"], **s)
        down(o["h"], d["w3"], o["off"], D=o["y"], **s)
        back(o["y"], o["rows"], d["w"], residual=d["x"], D=o["out"], **s)
        dback(d["dout"], o["y"], o["rows"], d["w"], dY=o["dy"], dweights=o["dw"], **s)
        ddown(o["dy"], o["h"], d["w3"], o["off"], dA=o["dh"], dB=o["dw3"], **s)
        dgate(o["dh"], o["xs"], d["w1"], o["off"], Z=o["z"], U=o["u"], dZ=o["dz"], dU=o["du"], dA=o["dxs"], dB=o["dw1"], **s)
        dup(o["du"], o["xs"], d["w2"], o["off"], dA=o["dxs2"], dB=o["dw2"], **s)
        dsort(o["dxs"], o["rows"], residual=d["dout"], D=o["dx1"], **s)
        dsort(o["dxs2"], o["rows"], residual=o["dx1"], D=o["dx"], **s)

    return host, call, new


@pytest.mark.parametrize("T,k,E,H,F", [(9, 2, 8, 64, 40), (300, 3, 5, 136, 264)])
def test_mixture_of_experts(T, k, E, H, F):
    """Forward and backward against 64-bit autograd of the same layer.  Every
    16-bit tensor on the way is off by half a step (2^-9 of its size at random,
    2^-8 at most), so the result's relative error in the 2-norm is at most the
    sum of its 2^-8 over the roundings in a row: 5 forward (xs is a copy; u, h,
    y, out and z's use), 9 for dx."""
    host, call, new = _layer(T, k, E, H, F, T)
    o = new()
    _say("case mixture", T, k, E, H, F)
    call(o)
    torch.cuda.synchronize()
    v = {n: (t.double().requires_grad_() if t.is_floating_point() else t) for n, t in host.items()}
    terms = []
    for t in range(T):
        row = v["x"][t]
        for j, e in enumerate(host["ids"][t].tolist()):
            if e >= 0:
                hidden = torch.nn.functional.silu(v["w1"][e] @ v["x"][t]) * (v["w2"][e] @ v["x"][t])
                row = row + v["w"][t, j] * (v["w3"][e] @ hidden)
        terms.append(row)
    out = torch.stack(terms)
    (out * host["dout"].double()).sum().backward()
    far = lambda got, want: float((ref.f64(got) - want).norm() / want.norm())  # noqa: E731
    assert far(o["out"], out.detach()) <= 5 * 2.0 ** -8
    for name, got, steps in (("w3", o["dw3"], 5), ("w1", o["dw1"], 7), ("w2", o["dw2"], 7), ("w", o["dw"], 4),
                             ("x", o["dx"], 9)):
        assert far(got, v[name].grad) <= steps * 2.0 ** -8, name


def test_streams_and_graphs():
    """The whole layer on two streams at once, and in two graphs replayed in
    turn, bit for bit as alone."""
    _, call, new = _layer(257, 3, 6, 128, 200, 5)
    _say("case streams and graphs")
    want = new()
    call(want)
    torch.cuda.synchronize()
    same = lambda o: all(torch.equal(o[n], want[n]) for n in want)  # noqa: E731
    outs = [new() for _ in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        call(o, streams[i % 2])
    torch.cuda.synchronize()
    assert all(map(same, outs))
    graphs = []
    for o in outs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(o)
        graphs.append(gr)
    for _ in range(3):
        for o in outs[:2]:
            for t in o.values():
                t.zero_()
        eager = new()
        for gr in graphs:
            gr.replay()
        call(eager)
        torch.cuda.synchronize()
        assert same(eager) and all(map(same, outs[:2]))


def test_refusals():
    R, E, N, K = 16, 4, 64, 64
    b = dict(dtype=torch.bfloat16, device="cuda")
    A, B, D, U = torch.zeros(R, K, **b), torch.zeros(E, N, K, **b), torch.zeros(R, N, **b), torch.zeros(R, N, **b)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    op = ge.ExpertLinear(R, E, N, K, mul=True)
    good = dict(A=A, B=B, offsets=off, D=D, U=U)
    op(**good)
    for bad in (dict(U=None), dict(B=B[:2]), dict(B=B.half()), dict(offsets=off.long()), dict(offsets=off[:2]), dict(D=A[:4]),
                dict(D=A), dict(Z=torch.zeros_like(D)), dict(bias=torch.zeros(E, N, device="cuda")), dict(A=A.cpu()),
                dict(B=torch.zeros(E, K, N, **b).transpose(1, 2)), dict(offsets=None)):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            op(**(good | bad))
    grad = ge.ExpertLinearGrad(R, E, N, K, act="silu", mul=True, da="bf16", db="f32", dbias="f32")
    t = lambda: torch.zeros(R, 64, **b)  # noqa: E731
    good = dict(dD=t(), A=t(), B=B, offsets=off, Z=t(), U=t(), dZ=t(), dU=t(), dA=t(),
                dB=torch.zeros(E, N, K, device="cuda"), dbias=torch.zeros(E, N, device="cuda"))
    grad(**good)
    for bad in (dict(Z=None), dict(dZ=None), dict(U=None), dict(dU=None), dict(A=None), dict(B=None), dict(dA=None),
                dict(dbias=None), dict(dU=good["dZ"]), dict(dU=good["dD"]), dict(dZ=good["U"]), dict(dZ=good["A"]),
                dict(dA=good["A"]), dict(offsets=None), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, ge.GemmEpiError)):
            grad(**(good | bad))


def test_far_weights_and_rows():
    """Weights of more than 4 GiB in all, and rows that begin more than 4 GiB into A
    and D, through the few-row kernels and the tiles."""
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("less than 64 GiB of device memory free")
    g = torch.Generator().manual_seed(4)
    E, N, K = 40, 8192, 8192  # 5.4 GB of bf16
    last = _draw(g, N, K, torch.bfloat16, K ** -0.5)
    B = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    B[E - 1] = last.cuda()
    for R in (3, 100):
        A = _draw(g, R, K, torch.bfloat16)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = R
        D = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
        op = ge.ExpertLinear(R, E, N, K)
        _say("case far weights", R, op.plan["name"])
        op(A.cuda(), B, off, D=D)
        cols = slice(N - 64, N)
        dr, _, S = ref.linear(A, last[cols])
        ref.check("D", D[:, cols], dr, (K + 4) * ref.U * S + ref.half_step(dr.abs() + K * ref.U * S, torch.bfloat16))
    del B
    R, E, N, K, ld = 1200, 3, 64, 64, 2 << 20  # 4 MiB between rows: 5 GB
    big = torch.zeros(R, ld, dtype=torch.bfloat16, device="cuda")
    A, B = _draw(g, R, K, torch.bfloat16), _draw(g, E * N, K, torch.bfloat16).view(E, N, K)
    view = big[:, :K]
    view.copy_(A)
    out = big[:, 64:64 + N]
    off = [0, 5, 1000, R]
    op = ge.ExpertLinear(R, E, N, K, lda=ld, ldd=ld)
    _say("case far rows", op.plan["name"])
    op(view, B.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"), D=out)
    for e in range(E):
        at = slice(off[e], off[e + 1])
        dr, _, S = ref.linear(A[at], B[e])
        ref.check("D", out[at], dr, (K + 4) * ref.U * S + ref.half_step(dr.abs() + K * ref.U * S, torch.bfloat16))
