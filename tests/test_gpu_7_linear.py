"""The 16-bit products (moe_fp4_linear, moe_fp4_linear_backward) against fp64,
dense and grouped, with the bounds that tests/linear_ref.py derives."""
import math

import pytest
import torch

from fp4_routed_expert_router_b200 import moe
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    c = moe.Context(128, 128, 1, 1, 1, 1, 1)
    yield c
    c.close()


def _ok(ctx):
    torch.cuda.synchronize()
    assert ctx.last_error()[0] == moe.OK


def _rand(*shape, dtype=BF, scale=1.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + math.prod(shape) % 999983)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _padded(t, pad):
    """The same values in rows that are `pad` elements further apart (the gap holds NaN)."""
    if not pad:
        return t
    big = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), math.nan, dtype=t.dtype, device=t.device)
    big[..., :t.shape[-1]] = t
    return big[..., :t.shape[-1]]


# rows, K, N, act, type, y type, bias type, residual type, padding of the rows
FORWARD = [
    (1, 1, 1, "none", BF, None, None, None, 0),
    (1, 5120, 384, "none", BF, F, F, None, 0),
    (3, 8, 5, "relu", HF, None, HF, F, 0),
    (17, 64, 16, "silu", BF, None, BF, BF, 0),
    (64, 2304, 640, "swiglu", BF, None, None, None, 0),
    (64, 5120, 384, "none", BF, F, F, None, 8),
    (129, 130, 131, "gelu", HF, None, F, HF, 0),
    (128, 128, 128, "none", BF, None, None, None, 0),
    (129, 136, 136, "swiglu", HF, HF, HF, None, 8),
    (257, 520, 264, "silu", BF, F, None, F, 0),
    (333, 1001, 517, "gelu", HF, None, HF, HF, 0),
    (300, 1001, 130, "swiglu", BF, None, BF, BF, 3),
    (1000, 2304, 1288, "none", BF, BF, None, F, 0),
    (520, 4096, 520, "none", HF, F, None, None, 0),
    (2050, 328, 777, "relu", BF, None, F, BF, 8),
]


@pytest.mark.parametrize("R,K,N,act,dt,out,bt,rt,pad", FORWARD)
def test_forward(ctx, R, K, N, act, dt, out, bt, rt, pad):
    x = _padded(_rand(R, K, dtype=dt, seed=1), pad)
    two = act == "swiglu"
    w = _padded(_rand(N, K, dtype=dt, scale=K ** -0.5, seed=2), pad)
    wu = _padded(_rand(N, K, dtype=dt, scale=K ** -0.5, seed=3), pad) if two else None
    b = _rand(N, dtype=bt, seed=4) if bt else None
    bu = _rand(N, dtype=bt, seed=5) if bt and two else None
    r = _padded(_rand(R, N, dtype=rt, seed=6), pad) if rt else None
    y, z, zu = ctx.linear(x, w, w_up=wu, bias=b, bias_up=bu, act=act, residual=r, out_dtype=out, save=True)
    y2 = ctx.linear(x, w, w_up=wu, bias=b, bias_up=bu, act=act, residual=r, out_dtype=out)
    _ok(ctx)
    assert y.dtype == (out or dt) and torch.equal(y, y2)
    want, err, zr, ur, ze, ue = ref.forward(x, w, wu, b, bu, act, out=y.dtype)
    if r is not None:
        want = want + r.double()
        err = err + 2 * ref.CUT * want.abs()
    ref.close(y, want, err, "y")
    ref.close(z, zr, ze, "z")
    if two:
        ref.close(zu, ur, ue, "z_up")


# counts of each group's rows, K, N, act, type, y type, bias type
GROUPS = [
    ([0, 3, 0, 1, 5], 64, 48, "none", BF, None, None),
    ([1], 256, 128, "silu", BF, None, F),
    ([0, 0, 0], 64, 64, "none", BF, None, None),
    ([130, 0, 1, 255, 256, 2], 200, 136, "swiglu", HF, None, HF),
    ([70, 9, 0, 300], 1001, 131, "gelu", BF, None, BF),
    ([5] * 64, 2304, 256, "none", BF, F, None),
    ([0] * 40 + [600] + [0] * 23, 328, 392, "swiglu", BF, None, None),
]


def _grouping(counts, seed, gather=True, scatter=True, tokens=None):
    g = torch.Generator().manual_seed(seed)
    R = sum(counts)
    offs = [0]
    for c in counts:
        offs.append(offs[-1] + c)
    tokens = tokens or max(1, R // 2)
    xr = torch.randint(0, tokens, (R,), generator=g).int().cuda() if gather else None
    yr = torch.randperm(R, generator=g).int().cuda() if scatter else None
    return offs, torch.tensor(offs, dtype=torch.int32, device="cuda"), xr, yr, (tokens if gather else R), R


@pytest.mark.parametrize("index", [False, True])
@pytest.mark.parametrize("counts,K,N,act,dt,out,bt", GROUPS)
def test_grouped_forward(ctx, counts, K, N, act, dt, out, bt, index):
    offs, od, xr, yr, xt, R = _grouping(counts, 7, index, index)
    E, two = len(counts), act == "swiglu"
    x = _rand(max(xt, 1), K, dtype=dt, seed=11)[:xt]
    w = _rand(E, N, K, dtype=dt, scale=K ** -0.5, seed=12)
    wu = _rand(E, N, K, dtype=dt, scale=K ** -0.5, seed=13) if two else None
    b = _rand(E, N, dtype=bt, seed=14) if bt else None
    bu = _rand(E, N, dtype=bt, seed=15) if bt and two else None
    y, z, zu = ctx.grouped_linear(x, w, od, w_up=wu, bias=b, bias_up=bu, act=act, x_rows=xr, y_rows=yr,
                                  out_dtype=out, save=True)
    _ok(ctx)
    want, err, zr, ur, ze, ue = ref.forward(x, w, wu, b, bu, act, offs, xr, y.dtype)
    got = y if yr is None else y[yr.long()]
    ref.close(got, want, err, "y")
    ref.close(z, zr, ze, "z")
    if two:
        ref.close(zu, ur, ue, "z_up")


def test_rows_outside_the_groups_are_left(ctx):
    K, N, R = 72, 40, 50
    od = torch.tensor([7, 20, 20, 41], dtype=torch.int32, device="cuda")
    x, w = _rand(R, K, seed=1), _rand(3, N, K, seed=2)
    x[:7] = math.nan
    x[41:] = math.inf
    y = torch.full((R, N), 3.0, dtype=BF, device="cuda")
    ctx.grouped_linear(x, w, od, y=y)
    _ok(ctx)
    assert bool((y[:7] == 3).all()) and bool((y[41:] == 3).all())
    want, err, *_ = ref.forward(x, w, offsets=[7, 20, 20, 41])
    ref.close(y[7:41], want[7:41], err[7:41])
    dy = _rand(R, N, seed=3)
    dy[:7] = math.nan
    dx = torch.full((R, K), 5.0, dtype=BF, device="cuda")
    g = ctx.grouped_linear_backward(dy, x, w, od, dx=dx, need_db=True)
    _ok(ctx)
    assert bool((dx[:7] == 5).all()) and bool((dx[41:] == 5).all())
    (dxr, dxe), dw, db = ref.backward(dy, x, w, offsets=[7, 20, 20, 41])
    ref.close(dx[7:41], dxr[7:41], dxe[7:41], "dx")
    ref.close(g.dw, *dw[0], "dw")
    ref.close(g.db, *db[0], "db")
    assert bool((g.dw[1] == 0).all()) and bool((g.db[1] == 0).all())


# rows, K, N, act, type, dy type, dw type, padding
BACKWARD = [
    (1, 1, 1, "none", BF, None, None, 0),
    (5, 8, 3, "relu", HF, None, None, 0),
    (129, 256, 131, "silu", HF, None, None, 0),
    (128, 128, 128, "none", BF, None, F, 0),
    (300, 520, 384, "none", BF, F, None, 0),
    (1000, 640, 384, "none", BF, None, F, 0),
    (257, 264, 136, "swiglu", BF, None, None, 8),
    (333, 131, 517, "gelu", BF, F, None, 0),
    (70, 1001, 66, "swiglu", HF, None, None, 3),
    (2500, 200, 72, "silu", BF, None, None, 0),
]


@pytest.mark.parametrize("R,K,N,act,dt,dyt,dwt,pad", BACKWARD)
def test_backward(ctx, R, K, N, act, dt, dyt, dwt, pad):
    two = act == "swiglu"
    x = _padded(_rand(R, K, dtype=dt, seed=1), pad)
    w = _padded(_rand(N, K, dtype=dt, scale=K ** -0.5, seed=2), pad)
    wu = _padded(_rand(N, K, dtype=dt, scale=K ** -0.5, seed=3), pad) if two else None
    dy = _padded(_rand(R, N, dtype=dyt or dt, scale=0.3, seed=4), pad)
    z = _padded(_rand(R, N, dtype=dt, seed=5), pad) if act != "none" else None
    zu = _padded(_rand(R, N, dtype=dt, seed=6), pad) if two else None
    g = ctx.linear_backward(dy, x, w, w_up=wu, z=z, z_up=zu, act=act, need_db=True, dw_dtype=dwt)
    _ok(ctx)
    out = g.dw.dtype
    (dx, dxe), dw, db = ref.backward(dy, x, w, wu, z, zu, act, out=out)
    (_, dxe16), _, _ = ref.backward(dy, x, w, wu, z, zu, act, out=g.dx.dtype)
    ref.close(g.dx, dx, dxe16, "dx")
    ref.close(g.dw, *dw[0], "dw")
    ref.close(g.db, *db[0], "db")
    if two:
        ref.close(g.dw_up, *dw[1], "dw_up")
        ref.close(g.db_up, *db[1], "db_up")
    # the same bits again, and each gradient alone
    h = ctx.linear_backward(dy, x, w, w_up=wu, z=z, z_up=zu, act=act, need_dw=False)
    k = ctx.linear_backward(dy, x, w, w_up=wu, z=z, z_up=zu, act=act, need_dx=False, dw_dtype=dwt)
    m = ctx.linear_backward(dy, x, w, w_up=wu, z=z, z_up=zu, act=act, need_dx=False, need_dw=False, need_db=True)
    _ok(ctx)
    assert torch.equal(h.dx, g.dx) and torch.equal(k.dw, g.dw) and torch.equal(m.db, g.db)
    assert h.dw is None and k.dx is None and m.dx is None
    # accumulation over micro-batches
    acc = [t.clone() if t is not None else None for t in (g.dw, g.dw_up, g.db, g.db_up)]
    ctx.linear_backward(dy, x, w, w_up=wu, z=z, z_up=zu, act=act, need_dx=False, need_db=True, dw=acc[0],
                        dw_up=acc[1], db=acc[2], db_up=acc[3], accumulate=True)
    _ok(ctx)
    ref.close(acc[0], 2 * dw[0][0], 2 * dw[0][1] + ref.rounding(dw[0][0], out), "accumulated dw")
    ref.close(acc[2], 2 * db[0][0], 2 * db[0][1] + ref.rounding(db[0][0], F), "accumulated db")


@pytest.mark.parametrize("index", [False, True])
@pytest.mark.parametrize("counts,K,N,act,dt,out,bt", GROUPS)
def test_grouped_backward(ctx, counts, K, N, act, dt, out, bt, index):
    offs, od, xr, yr, xt, R = _grouping(counts, 9, index, index)
    E, two = len(counts), act == "swiglu"
    x = _rand(max(xt, 1), K, dtype=dt, seed=11)[:xt]
    w = _rand(E, N, K, dtype=dt, scale=K ** -0.5, seed=12)
    wu = _rand(E, N, K, dtype=dt, scale=K ** -0.5, seed=13) if two else None
    dy = _rand(max(R, 1), N, dtype=dt, scale=0.3, seed=14)[:R]
    z = _rand(max(R, 1), N, dtype=dt, seed=15)[:R] if act != "none" else None
    zu = _rand(max(R, 1), N, dtype=dt, seed=16)[:R] if two else None
    g = ctx.grouped_linear_backward(dy, x, w, od, w_up=wu, z=z, z_up=zu, act=act, x_rows=xr, y_rows=yr, dx_rows=yr,
                                    need_db=True)
    _ok(ctx)
    (dx, dxe), dw, db = ref.backward(dy, x, w, wu, z, zu, act, offs, xr, yr, out=g.dx.dtype)
    ref.close(g.dx if yr is None else g.dx[yr.long()], dx, dxe, "dx")
    ref.close(g.dw, *dw[0], "dw")
    ref.close(g.db, *db[0], "db")
    if two:
        ref.close(g.dw_up, *dw[1], "dw_up")
        ref.close(g.db_up, *db[1], "db_up")


def test_no_rows(ctx):
    x, w = _rand(4, 64)[:0], _rand(32, 64, seed=1)
    assert ctx.linear(x, w).shape == (0, 32)
    g = ctx.linear_backward(_rand(4, 32)[:0], x, w, need_db=True)
    _ok(ctx)
    assert g.dx.shape == (0, 64) and bool((g.dw == 0).all()) and bool((g.db == 0).all())
    keep = torch.full_like(w, 2.0)
    ctx.linear_backward(_rand(4, 32)[:0], x, w, dw=keep, accumulate=True, need_dx=False)
    _ok(ctx)
    assert bool((keep == 2).all())


def test_bad_indices_are_latched_and_stay_inside(ctx):
    K, N, R = 64, 64, 40
    x, w = _rand(R, K, seed=1), _rand(2, N, K, seed=2)
    od = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    xr = torch.arange(R, dtype=torch.int32, device="cuda")
    xr[3], xr[30] = -1, R
    y = ctx.grouped_linear(x, w, od, x_rows=xr)
    torch.cuda.synchronize()
    assert ctx.last_error()[0] == moe.EINVAL
    assert bool((y[3] == 0).all()) and bool((y[30] == 0).all())
    good = ctx.grouped_linear(x, w, od)
    keep = [i for i in range(R) if i not in (3, 30)]
    assert torch.equal(y[keep], good[keep])
    yr = torch.arange(R, dtype=torch.int32, device="cuda")
    yr[5], yr[39] = 1 << 30, -7
    y = torch.full((R, N), 9.0, dtype=BF, device="cuda")
    ctx.grouped_linear(x, w, od, y_rows=yr, y=y)
    torch.cuda.synchronize()
    assert ctx.last_error()[0] == moe.EINVAL
    assert bool((y[5] == 9).all()) and bool((y[39] == 9).all())
    keep = [i for i in range(R) if i not in (5, 39)]
    assert torch.equal(y[keep], good[keep])
    for bad in ([0, 50, 40], [-4, 20, 40], [0, 20, 41]):    # only sound groups are computed
        y = torch.full((R, N), 9.0, dtype=BF, device="cuda")
        ctx.grouped_linear(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), y=y)
        torch.cuda.synchronize()
        assert ctx.last_error()[0] == moe.EINVAL
        for e in range(2):
            if 0 <= bad[e] <= bad[e + 1] <= R:
                lo, hi = bad[e], bad[e + 1]
                assert torch.equal(y[lo:hi], ctx.linear(x[lo:hi], w[e]))
    assert ctx.last_error()[0] == moe.OK
