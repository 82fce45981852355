"""Every tile kernel of the linear layer in its steady state: K of many K tiles
and a cut one, so the ring of stages turns over without guards; more tiles than
workgroups, so a workgroup enters the ring a second time; and plans whose last
round is cut into K slices behind whole tiles.  Also the backward's tiles over
long contractions.  Bounds: tests/linear_ref.py."""
import pytest
import torch

import beta_epilogue_amd as ge
import linear_ref as ref
from test_linear_gpu import ACTS, Out, _draw, _say, run_grad

pytestmark = pytest.mark.gpu

NAMES = ge.linear_variant_names()[:-1]
M = 300


def _f64(t):
    """Stored values as float64 on the GPU."""
    return t.float().double()


def _bounds(d, z, S, K, ab, dtype, fp8):
    """ref.linear_bounds on the device, with |residual| <= |d| + |z|."""
    acc = 1e-3 if fp8 else (2 * ref.U if ab == "i8" else K * ref.U)
    ez = (acc + 4 * ref.U) * S
    return ez, 1.13 * ez + z.abs() * 2.0 ** -21 + ref.U * (d.abs() + 2 * z.abs())


def _run(name, N, K, act, splits, want_split):
    ab = name.split("_")[1]
    d = "f32" if "f32" in name else {"f16": "f16"}.get(ab, "bf16")
    T, DT, scaled = ref.TORCH[ab], ref.TORCH[d], ab in ("e4m3", "i8")
    g = torch.Generator().manual_seed(K)
    A, B = _draw(g, M, K, T).cuda(), _draw(g, N, K, T, 1.0 if scaled else K ** -0.5).cuda()
    unit = K ** -0.5 * (1 / 1600.0 if ab == "i8" else 1.0)
    sa = (torch.rand(M, generator=g) + 0.5).cuda() if scaled else None
    sb = ((torch.rand(N, generator=g) + 0.5) * unit).cuda() if scaled else None
    bias, R = torch.randn(N, generator=g).cuda(), _draw(g, M, N, DT).cuda()
    op = ge.FusedLinear(M, N, K, ab=ab, d=d, act=act, bias="f32", residual=True, z=True, scale_a=scaled,
                        scale_b=scaled, variant=NAMES.index(name), splits=splits)
    plan = op.plan
    D, Z = Out(M, N, DT), Out(M, N, DT)
    _say("case", name, M, N, K, act, "tiles", plan["tiles"], "of", plan["grid"], "split", plan["split_tiles"], "in",
         plan["splits"])
    assert plan["tiles"] > plan["cus"]
    if want_split:
        assert plan["splits"] > 1 and 0 < plan["split_tiles"] < plan["tiles"]
    else:
        assert plan["splits"] == 1 and plan["grid"] < plan["tiles"]
    op(A, B, D=D.t, Z=Z.t, bias=bias, residual=R, scale_a=sa, scale_b=sb)
    torch.cuda.synchronize()
    assert D.intact() and Z.intact()
    a, b = _f64(A), _f64(B)
    if scaled:
        a, b = a * sa.double()[:, None], b * sb.double()[:, None]
    z = a @ b.T + bias.double()
    S = a.abs() @ b.abs().T + bias.double().abs()
    want = ref.act(z, act) + _f64(R)
    ez, ed = _bounds(want, z, S, K, ab, DT, ab == "e4m3" and d != "f32")
    for what, got, w, e in (("Z", Z.t, z, ez), ("D", D.t, want, ed)):
        off = ((_f64(got) - w).abs() - (e + w.abs().add(e) * ref.HALF_STEP[DT] + ref.TINY[DT])).max()
        assert float(off) <= 0, (what, float(off))
    op.close()


def _shape(name, whole_rounds):
    """(N, K tile) with a few tiles more than whole_rounds rounds of workgroups."""
    probe = ge.FusedLinear(M, 256, 256, ab=name.split("_")[1], d="f32" if "f32" in name else None, splits=1,
                           variant=NAMES.index(name)).plan
    slots = probe["cus"] * (2 if probe["lds_bytes"] <= 80 * 1024 else 1)
    if probe["lds_bytes"] * 3 <= 160 * 1024:
        slots = probe["cus"] * 3
    tiles_m = -(-M // probe["tile_m"])
    tiles_n = slots * whole_rounds // tiles_m + 2
    return (tiles_n - 1) * probe["tile_n"] + 8, probe["tile_k"]


@pytest.mark.parametrize("name", NAMES)
def test_long_k_and_second_items(name):
    N, bk = _shape(name, 1)
    _run(name, N, 13 * bk + 16, ACTS[NAMES.index(name) % 5], 1, False)


@pytest.mark.parametrize("name", NAMES)
def test_whole_tiles_then_k_slices(name):
    N, bk = _shape(name, 1)
    _run(name, N, 64 * bk + 16, ACTS[(NAMES.index(name) + 2) % 5], 0, True)


def test_large_rounds_in_slices():
    """The planner's own choice for a grid of several rounds and a rest."""
    for ab, d in (("bf16", "bf16"), ("i8", "bf16")):
        g = torch.Generator().manual_seed(7)
        m, n, k = 4352, 4352, 4096
        A, B = _draw(g, m, k, ref.TORCH[ab]).cuda(), _draw(g, n, k, ref.TORCH[ab], k ** -0.5 if ab == "bf16" else 1).cuda()
        op = ge.FusedLinear(m, n, k, ab=ab, d=d, act="silu", residual=True)
        R, D = (torch.randn(m, n, generator=g) * 64).bfloat16().cuda(), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        plan = op.plan
        _say("case", ab, plan)
        assert plan["splits"] > 1 and 0 < plan["split_tiles"] < plan["tiles"]
        alpha = 1.0 if ab == "bf16" else 2.0 ** -12
        op(A, B, D=D, residual=R, alpha=alpha)
        torch.cuda.synchronize()
        z = alpha * (_f64(A) @ _f64(B).T)
        S = alpha * (_f64(A).abs() @ _f64(B).abs().T)
        want = ref.act(z, "silu") + _f64(R)
        _, e = _bounds(want, z, S, k, ab, torch.bfloat16, False)
        assert float(((_f64(D) - want).abs() - (e + (want.abs() + e) * 2.0 ** -8)).max()) <= 2.0 ** -134


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("tile", [64, 128, 256])
def test_grad_long_contractions(tile, splits):
    """Contractions of 16 and more K tiles in both products; few items (the
    deep ring of 128x128 tiles) and more than two rounds."""
    run_grad(1100, 1032, 264, "bf16", "silu", da="bf16", db="f32", dbias="f32", db_in=True, tile=tile, splits=splits)
    run_grad(1544, 2088, 1288, "f16", "relu", da="f32", db="f16", dbias="f32", tile=tile, splits=splits)
