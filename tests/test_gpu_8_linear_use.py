"""The 16-bit products as they are used: sizes over the whole range, outputs in
place, far strides, streams, graphs, calls at once, refusals of the C call, a
wait that runs out, and a training step of a layer with routed and shared
experts against fp64 autograd."""
import ctypes
import math
import random

import pytest
import torch

from fp4_routed_expert_router_b200 import moe, synth
from tests import linear_ref as ref
from tests.gpu_helpers import Filled, check_routing, check_y, to_dev

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    c = moe.Context(128, 128, 1, 1, 1, 1, 1)
    yield c
    c.close()


def _ok(ctx):
    torch.cuda.synchronize()
    rc, msg = ctx.last_error()
    assert rc == moe.OK, msg


def _rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _log(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


@pytest.mark.parametrize("seed", range(24))
def test_sizes_over_the_range(ctx, seed):
    """Dense and grouped, forward and backward, at sizes that reach every tile shape."""
    r, g = random.Random(seed), _gen(seed)
    act = r.choice(["none", "relu", "silu", "gelu", "swiglu"])
    dt, out = r.choice([BF, HF]), r.choice([None, F])
    K, N, R = _log(r, 8, 4000), _log(r, 8, 2600), _log(r, 1, 3000)
    if r.random() < 0.7:
        K, N = max(8, K // 8 * 8), max(16, N // 16 * 16)
    E = r.choice([0, 0, 3, 17, 64])
    two = act == "swiglu"
    lead = (E,) if E else ()
    if E:
        cuts = sorted(r.choices(range(R + 1), k=E - 1))
        offs = [0] + cuts + [R]
        od = torch.tensor(offs, dtype=torch.int32, device="cuda")
        T = max(1, R // 2)
        xr = torch.randint(0, T, (R,), generator=g, device="cuda").int()
        yr = torch.randperm(R, generator=g, device="cuda").int()
    else:
        offs, T, xr, yr = None, R, None, None
    x = _rand(g, T, K, dtype=dt)
    w = _rand(g, *lead, N, K, dtype=dt, scale=K ** -0.5)
    wu = _rand(g, *lead, N, K, dtype=dt, scale=K ** -0.5) if two else None
    b = _rand(g, *lead, N, dtype=F) if r.random() < 0.5 else None
    kw = {"w_up": wu, "bias": b, "act": act, "out_dtype": out}
    if E:
        y = ctx.grouped_linear(x, w, od, x_rows=xr, y_rows=yr, **kw)
    else:
        y = ctx.linear(x, w, **kw)
    _ok(ctx)
    want, err, *_ = ref.forward(x, w, wu, b, None, act, offs, xr, y.dtype)
    ref.close(y if yr is None else y[yr.long()], want, err, "y")
    dy = _rand(g, R, N, dtype=dt, scale=0.3)
    z = _rand(g, R, N, dtype=dt) if act != "none" else None
    zu = _rand(g, R, N, dtype=dt) if two else None
    kw = {"w_up": wu, "z": z, "z_up": zu, "act": act, "need_db": True}
    if E:
        d = ctx.grouped_linear_backward(dy, x, w, od, x_rows=xr, y_rows=yr, dx_rows=yr, **kw)
    else:
        d = ctx.linear_backward(dy, x, w, **kw)
    _ok(ctx)
    (dx, dxe), dw, db = ref.backward(dy, x, w, wu, z, zu, act, offs, xr, yr, out=dt)
    ref.close(d.dx if yr is None else d.dx[yr.long()], dx, dxe, "dx")
    for got, (v, e) in zip((d.dw, d.dw_up) if two else (d.dw,), dw):
        ref.close(got, v, e, "dw")
    for got, (v, e) in zip((d.db, d.db_up) if two else (d.db,), db):
        ref.close(got, v, e, "db")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("R,K,N", [(5, 64, 40), (700, 520, 1032)])
def test_residual_in_place(ctx, R, K, N, dtype):
    g = _gen(1)
    x, w, y = _rand(g, R, K), _rand(g, N, K, scale=K ** -0.5), _rand(g, R, N, dtype=dtype)
    keep = y.clone()
    out = ctx.linear(x, w, residual=y, y=y)
    other = ctx.linear(x, w, residual=keep, out_dtype=dtype)
    _ok(ctx)
    assert out.data_ptr() == y.data_ptr() and torch.equal(y, other)
    want, err, *_ = ref.forward(x, w, out=dtype)
    want = want + keep.double()
    ref.close(y, want, err + 2 * ref.CUT * (want.abs() + keep.double().abs()))


def test_rows_far_apart(ctx):
    """Row and group strides whose byte offsets pass 32 bits, of inputs and outputs."""
    far = (1 << 31) + 64                       # elements
    big = torch.zeros(2 * far + 4096, dtype=BF, device="cuda")
    g = _gen(2)
    K, N = 72, 48
    x, w = _rand(g, 3, K), _rand(g, 2, N, K, scale=K ** -0.5)
    xs = big.as_strided((3, K), (far, 1))
    xs.copy_(x)
    near = ctx.linear(x, w[0])
    got = ctx.linear(xs, w[0])
    ys = big.as_strided((3, N), (far, 1), 1024)
    ctx.linear(x, w[0], y=ys)
    ws = big.as_strided((2, N, K), (far, K, 1), 2048 - 2048 % 8)
    ws.copy_(w)
    od = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    grouped = ctx.grouped_linear(x, w, od)
    grouped_far = ctx.grouped_linear(x, ws, od)
    dy = _rand(g, 3, N)
    d = ctx.grouped_linear_backward(dy, x, w, od)
    dws = big.as_strided((2, N, K), (far, K, 1), 2048 - 2048 % 8)
    e = ctx.grouped_linear_backward(dy, x, ws.clone(), od, dw=dws)
    _ok(ctx)
    assert torch.equal(near, got) and torch.equal(near, ys)
    assert torch.equal(grouped, grouped_far)
    assert torch.equal(d.dx, e.dx) and torch.equal(d.dw, dws)
    del big


def _layer(ctx, g, n, out):
    x, w, wu = _rand(g, n, 520), _rand(g, 264, 520, scale=0.05), _rand(g, 264, 520, scale=0.05)
    w2, res = _rand(g, 520, 264, scale=0.05), _rand(g, n, 520)

    def run(stream=None):
        h, z, zu = ctx.linear(x, w, w_up=wu, act="swiglu", save=True, stream=stream)
        y = ctx.linear(h, w2, residual=res, out_dtype=out, stream=stream)
        d = ctx.linear_backward(res, h, w2, stream=stream)
        e = ctx.linear_backward(d.dx, x, w, w_up=wu, z=z, z_up=zu, act="swiglu", need_db=True, stream=stream)
        return y, d.dw, e.dx, e.dw, e.dw_up, e.db, e.db_up

    return run


def test_streams_of_their_own_and_at_once(ctx):
    """Work on other streams than the current one, two of them at a time, with inputs freed right after the calls."""
    runs = [_layer(ctx, _gen(10 + i), n, F if i else None) for i, n in enumerate((37, 900))]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got = [r(stream=s) for r, s in zip(runs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    # inputs that die while the side stream still works
    s = streams[0]
    g = _gen(20)
    keep_x, keep_w = _rand(g, 600, 1001), _rand(g, 500, 1001, scale=0.03)
    want_y = ctx.linear(keep_x, keep_w)
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        x, w = keep_x.clone(), keep_w.clone()
        s.wait_stream(torch.cuda.current_stream())
        outs.append(ctx.linear(x, w, stream=s))
        del x, w
        junk = [torch.full((600, 1001), 3.0, dtype=BF, device="cuda") for _ in range(4)]
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(o, want_y) for o in outs)
    _ok(ctx)


def test_two_captured_graphs_replayed_at_once(ctx):
    runs = [_layer(ctx, _gen(30 + i), n, None) for i, n in enumerate((64, 700))]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            r()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(r())
        graphs.append((gr, s))
    for o in outs:
        for t in o:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for gr, s in graphs:
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    _ok(ctx)


def test_replay_with_other_groups(ctx):
    """A captured grouped call reads offsets and indices at replay."""
    g = _gen(40)
    E, K, N, R = 8, 136, 72, 96
    x, w = _rand(g, 50, K), _rand(g, E, N, K, scale=0.1)
    od = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    xr = torch.zeros(R, dtype=torch.int32, device="cuda")
    dy = _rand(g, R, N)
    s = torch.cuda.Stream()
    y = torch.zeros(R, N, dtype=BF, device="cuda")

    def call():
        ctx.grouped_linear(x, w, od, x_rows=xr, y=y)
        return ctx.grouped_linear_backward(dy, x, w, od, x_rows=xr, need_db=True)

    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        d = call()
    r = random.Random(4)
    for _ in range(4):
        offs = [0] + sorted(r.choices(range(R + 1), k=E - 1)) + [R]
        od.copy_(torch.tensor(offs, dtype=torch.int32))
        xr.copy_(torch.randint(0, 50, (R,), generator=torch.Generator().manual_seed(r.randrange(99))).int())
        gr.replay()
        _ok(ctx)
        want, err, *_ = ref.forward(x, w, offsets=offs, x_rows=xr)
        ref.close(y, want, err, "y")
        (dx, dxe), dw, db = ref.backward(dy, x, w, offsets=offs, x_rows=xr)
        ref.close(d.dx, dx, dxe, "dx")
        ref.close(d.dw, *dw[0], "dw")
        ref.close(d.db, *db[0], "db")


def test_values_that_are_not_finite_stay_in_their_rows(ctx):
    """NaN and infinities of one row or group reach that row and group only."""
    g = _gen(50)
    K, N = 136, 72
    x, w = _rand(g, 40, K), _rand(g, 3, N, K, scale=0.1)
    od = torch.tensor([0, 13, 13, 40], dtype=torch.int32, device="cuda")
    dy = _rand(g, 40, N)
    y0 = ctx.grouped_linear(x, w, od)
    d0 = ctx.grouped_linear_backward(dy, x, w, od, need_db=True)
    x2, dy2 = x.clone(), dy.clone()
    x2[20, 3], dy2[25, 5] = math.inf, math.nan
    y1 = ctx.grouped_linear(x2, w, od)
    d1 = ctx.grouped_linear_backward(dy2, x2, w, od, need_db=True)
    _ok(ctx)
    rest = [i for i in range(40) if i != 20]
    assert torch.equal(y0[rest], y1[rest]) and not bool(torch.isfinite(y1[20]).any())
    rest = [i for i in range(40) if i != 25]
    assert torch.equal(d0.dx[rest], d1.dx[rest]) and bool(torch.isnan(d1.dx[25]).all())
    for a, b in ((d0.dw, d1.dw), (d0.db, d1.db)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(torch.isnan(d1.db[2, 5])) and bool(torch.isnan(d1.dw[2, 5]).all())


def test_groups_without_any_row(ctx):
    """Rows that no group holds, and groups that hold none: y stays, gradients are zero."""
    g = _gen(55)
    x, w, dy = _rand(g, 9, 72), _rand(g, 4, 40, 72), _rand(g, 9, 40)
    od = torch.full((5,), 4, dtype=torch.int32, device="cuda")
    y = torch.full((9, 40), 2.0, dtype=BF, device="cuda")
    ctx.grouped_linear(x, w, od, y=y, x_rows=torch.full((9,), -1, dtype=torch.int32, device="cuda"))
    dw = torch.full_like(w, 3.0, dtype=F)
    d = ctx.grouped_linear_backward(dy, x, w, od, dx=y.new_full((9, 72), 6.0), need_db=True)
    ctx.grouped_linear_backward(dy, x, w, od, need_dx=False, dw=dw, accumulate=True)
    _ok(ctx)
    assert bool((y == 2).all()) and bool((d.dx == 6).all()) and bool((dw == 3).all())
    assert bool((d.dw == 0).all()) and bool((d.db == 0).all())


def test_bad_indices_in_the_backward_pass(ctx):
    g = _gen(60)
    K, N, R = 72, 40, 30
    x, w, dy = _rand(g, R, K), _rand(g, 2, N, K, scale=0.1), _rand(g, R, N)
    od = torch.tensor([0, 11, 30], dtype=torch.int32, device="cuda")
    good = torch.arange(R, dtype=torch.int32, device="cuda")
    bad = good.clone()
    bad[4], bad[20] = -3, R
    zx, zdy = x.clone(), dy.clone()
    zx[[4, 20]] = 0
    zdy[[4, 20]] = 0
    for kw, (xx, dd) in (({"x_rows": bad}, (zx, dy)), ({"y_rows": bad}, (x, zdy))):
        d = ctx.grouped_linear_backward(dy, x, w, od, need_db=True, **kw)
        torch.cuda.synchronize()
        assert ctx.last_error()[0] == moe.EINVAL
        e = ctx.grouped_linear_backward(dd, xx, w, od, need_db=True)
        _ok(ctx)
        assert torch.equal(d.dw, e.dw) and torch.equal(d.db, e.db)
        if "y_rows" in kw:
            assert torch.equal(d.dx, e.dx)
    dx = torch.full((R, K), 7.0, dtype=BF, device="cuda")
    ctx.grouped_linear_backward(dy, x, w, od, need_dw=False, dx_rows=bad, dx=dx)
    torch.cuda.synchronize()
    assert ctx.last_error()[0] == moe.EINVAL
    assert bool((dx[[4, 20]] == 7).all())


@pytest.mark.parametrize("graph", [False, True])
def test_micro_batches_one_after_the_other(ctx, graph):
    """Backward calls without a pause, whose kernels begin beside the ends of those before and whose scratch is the
    same memory each time, give the bits of calls that are waited for."""
    g = _gen(63)
    R, K, N, E, n = 70, 136, 72, 3, 12
    x, w = _rand(g, R, K), _rand(g, E, N, K, scale=0.1)
    od = torch.tensor([0, 33, 33, R], dtype=torch.int32, device="cuda")
    z = _rand(g, R, N)
    dys = [_rand(g, R, N) for _ in range(n)]

    def batches(dw, db, wait):
        dxs = []
        for dy in dys:
            d = ctx.grouped_linear_backward(dy, x, w, od, z=z, act="silu", dw=dw, db=db, need_db=True, accumulate=True)
            dxs.append(d.dx)
            if wait:
                torch.cuda.synchronize()
        return torch.stack(dxs)

    want_w, want_b = torch.zeros(E, N, K, device="cuda"), torch.zeros(E, N, device="cuda")
    want_x = batches(want_w, want_b, True)
    dw, db = torch.zeros_like(want_w), torch.zeros_like(want_b)
    if graph:
        rec = torch.cuda.CUDAGraph()
        with torch.cuda.graph(rec):
            dx = batches(dw, db, False)
        dw.zero_()
        db.zero_()
        rec.replay()
    else:
        dx = batches(dw, db, False)
    _ok(ctx)
    assert torch.equal(dx, want_x) and torch.equal(dw, want_w) and torch.equal(db, want_b)


def test_offsets_that_descend_are_latched(ctx):
    """No result is valid then, but the call ends, reports it and stays inside its tensors: here every second group is
    all rows, so that the groups' tiles together are many times what sound groups could have."""
    g = _gen(61)
    K, N, R, E, edge = 72, 40, 33, 64, 64
    x, w, dy = _rand(g, R, K), _rand(g, E, N, K, scale=0.1), _rand(g, R, N)
    od = torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    y, dx = (torch.full((R + 2 * edge, n), 5.0, dtype=BF, device="cuda") for n in (N, K))
    dw = torch.full((E + 2, N, K), 5.0, dtype=F, device="cuda")
    ctx.grouped_linear(x, w, od, y=y[edge:-edge])
    torch.cuda.synchronize()
    assert ctx.last_error()[0] == moe.EINVAL
    ctx.grouped_linear_backward(dy, x, w, od, dx=dx[edge:-edge], dw=dw[1:-1], need_db=True)
    torch.cuda.synchronize()
    assert ctx.last_error()[0] == moe.EINVAL
    for t in (y, dx):
        assert bool((t[:edge] == 5).all()) and bool((t[-edge:] == 5).all())
    assert bool((dw[0] == 5).all()) and bool((dw[-1] == 5).all())
    ctx.grouped_linear(x, w[:2], torch.tensor([0, 3, R], dtype=torch.int32, device="cuda"))
    _ok(ctx)


def test_a_row_wider_than_a_grid_of_copies(ctx):
    """An odd length, which is copied, of more 512-column blocks than a grid's second dimension has.  Whole numbers,
    whose products and sums are exact in every order."""
    K = 512 * 65535 + 81
    g = _gen(62)
    x, w = (torch.zeros(1, K, dtype=BF, device="cuda") for _ in range(2))
    at = torch.cat([torch.randint(K, (500,), generator=g, device="cuda"), torch.arange(K - 90, K, device="cuda")])
    x[0, at] = torch.randint(-8, 9, (590,), generator=g, device="cuda").to(BF)
    w[0, at] = torch.randint(-8, 9, (590,), generator=g, device="cuda").to(BF)
    y = ctx.linear(x, w, out_dtype=F)
    d = ctx.linear_backward(torch.full((1, 1), 3.0, dtype=BF, device="cuda"), x, w)
    _ok(ctx)
    assert y.item() == (x.double() * w.double()).sum().item()
    assert torch.equal(d.dx, 3 * w) and torch.equal(d.dw.to(BF), 3 * x)


def test_the_c_call_refuses(ctx):
    x = torch.ones(4, 64, dtype=BF, device="cuda")
    w = torch.ones(32, 64, dtype=BF, device="cuda")
    y = torch.full((4, 32), 5.0, dtype=BF, device="cuda")

    def args(**kw):
        a = moe.LinearArgs(rows=4, in_features=64, out_features=32, x=x.data_ptr(), w=w.data_ptr(), y=y.data_ptr())
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    bad = [dict(rows=-1), dict(rows=(1 << 30) + 1), dict(in_features=0), dict(out_features=0), dict(type=2), dict(type=7), dict(act=5),
           dict(act=-1), dict(act=4), dict(w_up=w.data_ptr()), dict(n_groups=1025, offsets=x.data_ptr()),
           dict(n_groups=2), dict(offsets=x.data_ptr()), dict(n_groups=-1), dict(x=None), dict(w=None), dict(y=None),
           dict(ldx=63), dict(ldw=-64), dict(ldy=31), dict(y_type=3), dict(bias=x.data_ptr(), bias_type=9),
           dict(residual=x.data_ptr(), residual_type=-1), dict(residual=x.data_ptr(), ld_residual=3),
           dict(z_up=x.data_ptr()), dict(bias_up=x.data_ptr()), dict(reserved=1), dict(x=x.data_ptr() + 1),
           dict(y=y.data_ptr() + 1), dict(bias=x.data_ptr() + 2, bias_type=moe.F32),
           dict(x_rows=x.data_ptr()), dict(y_rows=x.data_ptr()), dict(x_rows=x.data_ptr() + 2, x_total=4),
           dict(x_rows=x.data_ptr(), x_total=4),                      # scratch is missing
           dict(ldx=68, scratch=x.data_ptr(), scratch_bytes=100),     # too little of it
           dict(ldx=68, scratch=x.data_ptr() + 8, scratch_bytes=1 << 30),
           dict(n_groups=2, offsets=x.data_ptr(), w_group_stride=64)]
    for kw in bad:
        rc = ctx.lib.moe_fp4_linear(ctx.h, ctypes.byref(args(**kw)), None)
        assert rc == moe.EINVAL, kw
        assert ctx.last_error()[0] == moe.EINVAL
    assert ctx.lib.moe_fp4_linear(ctx.h, None, None) == moe.EINVAL
    ctx.last_error()

    def grads(**kw):
        a = moe.LinearGradArgs(rows=4, in_features=64, out_features=32, x=x.data_ptr(), w=w.data_ptr(),
                               dy=y.data_ptr(), dx=x.data_ptr(), dw=w.data_ptr())
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    bad = [dict(rows=-1), dict(type=2), dict(dy_type=1), dict(dx_type=5), dict(dw_type=5), dict(dy=None), dict(x=None),
           dict(w=None), dict(act=2), dict(act=4), dict(dw_up=w.data_ptr()), dict(db_up=w.data_ptr()),
           dict(lddy=31), dict(lddx=63), dict(lddw=63), dict(ldz=3), dict(reserved=2), dict(dx_rows=x.data_ptr()),
           dict(db=x.data_ptr() + 2), dict(n_groups=3), dict(dy_type=2), dict(y_rows=x.data_ptr(), y_total=4)]
    for kw in bad:
        rc = ctx.lib.moe_fp4_linear_backward(ctx.h, ctypes.byref(grads(**kw)), None)
        assert rc == moe.EINVAL, kw
        assert ctx.last_error()[0] == moe.EINVAL
    torch.cuda.synchronize()
    assert bool((y == 5).all()) and bool((x == 1).all()) and bool((w == 1).all())


def test_profile_names_the_kernels(ctx):
    g = _gen(70)
    x, w, dy = _rand(g, 65, 1001), _rand(g, 40, 1001, scale=0.03), _rand(g, 65, 40)
    ctx.set_profile(True)
    try:
        ctx.linear(x, w)
        ctx.linear_backward(dy, x, w, need_db=True)
        names = [n for n, ms in ctx.profile_read() if ms > 0]
    finally:
        ctx.set_profile(False)
    assert names == ["linear_pack", "linear", "linear_pack", "linear_dz", "linear_dx", "linear_dw"]


@pytest.mark.parametrize("R,K,N", [(2048, 5120, 2304), (16, 81920, 384)])
def test_wait_limit_runs_out_then_calls_work_again(ctx, R, K, N):
    """A pair of CTAs and a split sum whose waits give up after a microsecond: ETIMEOUT, and the context goes on.

    The epilogue waits for a whole sum and looks at the clock every 1.4 us or so, so the sum has to take many times
    that: 80 stages of a pair take about 30 us, 160 of each CTA of a split sum (18 KB each at no more than 120 GB/s an
    SM) at least 24 us.  (A split sum of 5,120 terms is over in 3 us: whether its wait runs out is chance.)"""
    g = _gen(80)
    x, w = _rand(g, R, K), _rand(g, N, K, scale=K ** -0.5)
    good = ctx.linear(x, w)
    _ok(ctx)
    ctx.set_wait_limit_us(1)
    try:
        ctx.linear(x, w)
        torch.cuda.synchronize()
        rc, msg = ctx.last_error()
        assert rc == moe.ETIMEOUT and "linear" in msg, (rc, msg)
    finally:
        ctx.set_wait_limit_us(0)
    for _ in range(2):
        y = ctx.linear(x, w)
        _ok(ctx)
        assert torch.equal(y, good)


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_training_step_of_a_layer_with_routed_and_shared_experts():
    """Router, routed 16-bit experts, shared expert and their gradients, chained as a layer uses them, against fp64
    autograd.  Every value passes at most eight roundings to bf16 on its way, each off by at most 2^-8 of it, and the
    sums of such values stay as near in norm: 8 * 2^-8."""
    T, H, I, E, k = 60, 256, 128, 16, 2
    ctx = moe.Context(H, I, E, k, 1, E, T)
    try:
        g = _gen(90)
        x, gate = _rand(g, T, H), _rand(g, E, H, scale=H ** -0.5)
        gb = _rand(g, E, dtype=F, scale=0.1)
        w1, w3, w2 = (_rand(g, E, *s, scale=s[1] ** -0.5) for s in ((I, H), (I, H), (H, I)))
        s1, s3, s2 = (_rand(g, *s, scale=s[1] ** -0.5) for s in ((I, H), (I, H), (H, I)))
        dout = _rand(g, T, H)
        # forward
        logits = ctx.linear(x, gate, bias=gb, out_dtype=F)
        r = ctx.route(0, logits)
        token = r.perm // k
        h, z, zu = ctx.grouped_linear(x, w1, r.offsets, w_up=w3, act="swiglu", x_rows=token, save=True)
        o = ctx.grouped_linear(h, w2, r.offsets, y_rows=r.perm, out_dtype=F)
        y = ctx.combine(o, r.weights)
        hs, zs, zsu = ctx.linear(x, s1, w_up=s3, act="swiglu", save=True)
        out = ctx.linear(hs, s2, residual=y, out_dtype=F)
        # backward
        ds = ctx.linear_backward(dout, hs, s2)
        d1 = ctx.linear_backward(ds.dx, x, s1, w_up=s3, z=zs, z_up=zsu, act="swiglu")
        do = (r.weights.reshape(-1, 1) * dout.float().repeat_interleave(k, 0)).to(BF)
        d2 = ctx.grouped_linear_backward(do, h, w2, r.offsets, y_rows=r.perm)
        rows = torch.empty(T * k, H, dtype=F, device="cuda")
        d3 = ctx.grouped_linear_backward(d2.dx, x, w1, r.offsets, w_up=w3, z=z, z_up=zu, act="swiglu", x_rows=token,
                                         dx_rows=r.perm, dx=rows)
        dxr = ctx.combine(rows, torch.ones(T, k, device="cuda"))
        dw = (o.reshape(T, k, H) * dout.float()[:, None]).sum(-1)              # d loss / d router weight
        p = r.weights
        dsel = p * (dw - (p * dw).sum(1, keepdim=True))                        # through the softmax over the chosen
        dlogits = torch.zeros(T, E, device="cuda").scatter_(1, r.ids.long(), dsel)
        dg = ctx.linear_backward(dlogits, x, gate, need_db=True)
        torch.cuda.synchronize()
        rc, msg = ctx.last_error()
        assert rc == moe.OK, msg
        dx = dxr.double() + d1.dx.double() + dg.dx.double()
        # fp64 autograd of the same layer with the same choice of experts
        P = [t.double().requires_grad_() for t in (x, gate, gb, w1, w3, w2, s1, s3, s2)]
        X, G, B, W1, W3, W2, S1, S3, S2 = P
        sel = (X @ G.T + B).gather(1, r.ids.long())
        pw = torch.softmax(sel, 1)
        silu = torch.nn.functional.silu
        Y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            e = r.ids[:, j].long()
            a = silu(torch.einsum("th,tih->ti", X, W1[e])) * torch.einsum("th,tih->ti", X, W3[e])
            Y = Y + pw[:, j:j + 1] * torch.einsum("ti,thi->th", a, W2[e])
        Y = Y + (silu(X @ S1.T) * (X @ S3.T)) @ S2.T
        Y.backward(dout.double())
        tol = 8 * 2.0 ** -8
        got = [dx, dg.dw, dg.db, d3.dw, d3.dw_up, d2.dw, d1.dw, d1.dw_up, ds.dw]
        assert _rel(out, Y.detach()) < tol
        for name, a, t in zip("x gate bias w1 w3 w2 s1 s3 s2".split(), got, P):
            assert _rel(a, t.grad) < tol, name
    finally:
        ctx.close()


@pytest.mark.parametrize("T", [1, 4, 33, 130])
def test_fp4_layer_with_its_router_and_a_shared_expert(T):
    """The FP4 layer between this library's own router product and shared expert, without a wait in between and in a
    replayed graph: the bits of calls that are waited for one by one, the routed part within its bar of the oracle, the
    shared part of fp64.  There h is rounded to bf16 once (2^-8 of it at most) and sums of its values stay as near in
    norm; 2 * 2^-8 leaves as much again for the activation and the fp32 sums."""
    wl = synth.WORKLOADS["tiny"]
    f = Filled(wl, max_tokens=256, from_host=True)
    ctx = f.ctx
    try:
        H, I, E = wl.hidden, wl.inter, wl.n_experts
        g = _gen(70 + T)
        gate, gb = _rand(g, E, H, scale=H ** -0.5), _rand(g, E, dtype=F, scale=0.1)
        s1, s3, s2 = (_rand(g, *s, scale=s[1] ** -0.5) for s in ((I, H), (I, H), (H, I)))
        xs = [synth.gen_x(wl.seed, T, H, 5000 + i) for i in range(4)]
        x = to_dev(xs[0])

        def layer(wait=False):
            step = torch.cuda.synchronize if wait else (lambda: None)
            logits = ctx.linear(x, gate, bias=gb, out_dtype=F)
            step()
            r, y = ctx.route_forward(0, logits, x)
            step()
            h = ctx.linear(x, s1, w_up=s3, act="swiglu")
            step()
            return logits, r, y, ctx.linear(h, s2, residual=y, out_dtype=F)

        want = []
        for v in xs:
            x.copy_(to_dev(v))
            logits, r, y, out = layer(wait=True)
            _ok(ctx)
            ids, w = check_routing(r, logits.cpu().numpy(), wl.top_k, E)
            check_y(y.cpu().numpy(), f.oracle_y(0, v, ids, w, range(T)))
            X = x.view(BF).double()
            shared = (torch.nn.functional.silu(X @ s1.double().T) * (X @ s3.double().T)) @ s2.double().T
            assert _rel(out.double() - y.double(), shared) < 2 * 2.0 ** -8
            want.append((logits.clone(), y.clone(), out.clone()))
        for v, (a, b, c) in zip(xs, want):
            x.copy_(to_dev(v))
            logits, _, y, out = layer()
            _ok(ctx)
            assert torch.equal(logits, a) and torch.equal(y, b) and torch.equal(out, c)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            logits, _, y, out = layer()
        for v, (a, b, c) in zip(xs * 3, want * 3):
            x.copy_(to_dev(v))
            graph.replay()
            assert torch.equal(logits, a) and torch.equal(y, b) and torch.equal(out, c)
        _ok(ctx)
    finally:
        f.close()
