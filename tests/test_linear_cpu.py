"""Host-side checks of the 16-bit products (no GPU): the binding's structs match
the header, refusals before any launch, scratch sizes, the packed row layout,
launch plans against the B200 limits, and the fp64 formulas the GPU tests use
against central differences."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest
import torch

from fp4_routed_expert_router_b200 import build as pkg_build
from fp4_routed_expert_router_b200 import moe
from tests import linear_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp4_routed_expert_router_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return moe.load()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
@pytest.mark.parametrize("struct,name", [(moe.LinearArgs, "moe_fp4_linear_args"),
                                         (moe.LinearGradArgs, "moe_fp4_linear_grads")])
def test_structs_match_the_header(tmp_path, struct, name):
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include "moe_fp4.h"\n#include <stdio.h>\nint main(void) {\n' +
                   "".join(f'    printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) +
                   f'    printf("%zu\\n", sizeof({name}));\n    return 0;\n}}\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]
    # and no field of the header is missing
    text = open(os.path.join(ROOT, "include", "moe_fp4.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    declared = [v.strip(" *") for line in body.split(";") if line.strip()
                for v in re.sub(r"^\s*(const\s+)?\w+\s+", "", line.strip()).split(",")]
    assert declared == fields


def test_null_context_is_refused(lib):
    assert lib.moe_fp4_linear(None, ctypes.byref(moe.LinearArgs()), None) == moe.EINVAL
    assert lib.moe_fp4_linear_backward(None, ctypes.byref(moe.LinearGradArgs()), None) == moe.EINVAL
    assert lib.moe_fp4_linear_scratch(None) == 0
    assert lib.moe_fp4_linear_backward_scratch(None) == 0


def _up(n, m):
    return (n + m - 1) // m * m


def test_scratch_sizes(lib):
    def fwd(rows, K, N, x=4096, w=4096, groups=0, gather=0, **kw):
        a = moe.LinearArgs(rows=rows, in_features=K, out_features=N, n_groups=groups, x=x, w=w, **kw)
        if gather:
            a.x_rows = 4096
        return lib.moe_fp4_linear_scratch(ctypes.byref(a))

    assert fwd(100, 5120, 384) == 0                                   # everything as it lies
    assert fwd(100, 5120, 384, gather=1) == _up(100 * 5120 * 2, 256)   # a gathered x
    assert fwd(100, 5120, 384, x=4098) == _up(100 * 5120 * 2, 256)     # a misaligned x
    assert fwd(100, 5120, 384, ldx=5124) == _up(100 * 5120 * 2, 256)   # rows of x off the 16-byte grid
    assert fwd(3, 1001, 7) == _up(3 * 1008 * 2, 256) + _up(7 * 1008 * 2, 256)
    assert fwd(3, 1001, 7, ldx=1008, ldw=1008) == 0
    assert fwd(3, 64, 7, groups=5, offsets=4096) == 0
    assert fwd(3, 64, 7, groups=5, offsets=4096, w_group_stride=450) == _up(5 * 7 * 64 * 2, 256)
    assert fwd(0, 1001, 7) == 0

    def bwd(rows, K, N, act=0, groups=0, dx=4096, dw=4096, **kw):
        a = moe.LinearGradArgs(rows=rows, in_features=K, out_features=N, act=act, n_groups=groups, x=4096, w=4096,
                               dy=4096, dx=dx, dw=dw, **kw)
        return lib.moe_fp4_linear_backward_scratch(ctypes.byref(a))

    assert bwd(50, 64, 32) == 0                                        # dy serves as dz
    assert bwd(50, 64, 32, act=2) == _up(50 * 32 * 2, 256)
    assert bwd(50, 64, 32, dy_type=moe.F32) == _up(50 * 32 * 2, 256)
    assert bwd(50, 64, 33) == _up(50 * 40 * 2, 256)                    # rows of 33 values are not aligned
    assert bwd(50, 64, 32, act=4, w_up=4096, dw_up=4096) == 2 * _up(50 * 32 * 2, 256)
    rows = (50 + 16 * 4 + 31) // 16 * 16                               # packed: dz and x
    assert bwd(50, 64, 32, groups=4, offsets=4096) == _up(rows * 32 * 2, 256) + _up(rows * 64 * 2, 256)
    assert bwd(50, 64, 32, groups=4, offsets=4096, dw=None) == 0


# ------------------------------------------------------------------ refusals of the binding
class _NoLib:
    """A library none of whose calls may be reached."""

    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


@pytest.fixture
def ctx():
    """A context object whose device is the CPU's (-1), to reach the checks without a GPU."""
    c = moe.Context.__new__(moe.Context)
    c.lib, c.device, c.h = _NoLib(), -1, None
    return c


def _x(*s, dtype=BF):
    return torch.zeros(*s, dtype=dtype)


def _refused(f, *words):
    with pytest.raises(moe.MoeError) as e:
        f()
    assert e.value.status == moe.EINVAL
    for w in words:
        assert w in str(e.value), str(e.value)


def test_linear_refusals(ctx, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(moe, "_raw_stream", lambda d: 0)
    x, w = _x(4, 64), _x(32, 64)
    _refused(lambda: ctx.linear(x, _x(32, 63)), "x has shape")
    _refused(lambda: ctx.linear(x, _x(32, 64, dtype=HF)), "x has type")
    _refused(lambda: ctx.linear(x.float(), w.float()), "w has type")
    _refused(lambda: ctx.linear(_x(64), w), "x is not a tensor")
    _refused(lambda: ctx.linear(x, _x(2, 32, 64)), "w has shape")
    _refused(lambda: ctx.linear(x, _x(0, 64)), "w has shape")
    _refused(lambda: ctx.linear(x, w, act="tanh"), "tanh")
    _refused(lambda: ctx.linear(x, w, act="swiglu"), "w_up")
    _refused(lambda: ctx.linear(x, w, w_up=w), "w_up")
    _refused(lambda: ctx.linear(x, w, w_up=_x(32, 66)[:, :64], act="swiglu"), "strides")
    _refused(lambda: ctx.linear(x, w, w_up=_x(31, 64), act="swiglu"), "w_up has shape")
    _refused(lambda: ctx.linear(x, w, bias=_x(31)), "bias")
    _refused(lambda: ctx.linear(x, w, bias=_x(64)[::2]), "bias")
    _refused(lambda: ctx.linear(x, w, bias_up=_x(32)), "bias_up")
    _refused(lambda: ctx.linear(x, w, w_up=w, act="swiglu", bias=_x(32), bias_up=_x(32, dtype=F)), "bias")
    _refused(lambda: ctx.linear(x, w, residual=_x(4, 31)), "residual has shape")
    _refused(lambda: ctx.linear(x, w, residual=_x(4, 32).double()), "residual has type")
    _refused(lambda: ctx.linear(x, w, residual=_x(32, 4).t()), "contiguous")
    _refused(lambda: ctx.linear(x, w, y=_x(3, 32)), "y has shape")
    _refused(lambda: ctx.linear(x, w, y=_x(1, 32).expand(4, 32)), "overlap")
    _refused(lambda: ctx.linear(x, w, y=_x(4, 32), out_dtype=F), "out_dtype")
    _refused(lambda: ctx.linear(x, w, out_dtype=torch.float64), "out_dtype")
    _refused(lambda: ctx.linear([1.0], w), "x is not a tensor")
    _refused(lambda: ctx.linear(x.expand(4, 64)[:1].expand(4, 64), w), "overlap")


def test_grouped_refusals(ctx):
    x, w = _x(6, 64), _x(3, 32, 64)
    od = torch.zeros(4, dtype=torch.int32)
    ix = torch.zeros(6, dtype=torch.int32)
    _refused(lambda: ctx.grouped_linear(x, _x(32, 64), od), "w has shape")
    _refused(lambda: ctx.grouped_linear(x, w, od[:3]), "offsets")
    _refused(lambda: ctx.grouped_linear(x, w, od.long()), "offsets")
    _refused(lambda: ctx.grouped_linear(x, w, torch.zeros(8, dtype=torch.int32)[::2]), "offsets")
    _refused(lambda: ctx.grouped_linear(x, w, od, x_rows=ix.long()), "x_rows")
    _refused(lambda: ctx.grouped_linear(x, w, od, x_rows=ix.view(2, 3)), "x_rows")
    _refused(lambda: ctx.grouped_linear(x, w, od, y_rows=ix[:5]), "y_rows")
    _refused(lambda: ctx.grouped_linear(x, w, od, bias=_x(32)), "bias")
    _refused(lambda: ctx.grouped_linear(x, _x(3, 1, 64).expand(3, 32, 64), od), "overlap")
    _refused(lambda: ctx.grouped_linear(x, _x(1, 32, 64).expand(3, 32, 64), od), "overlap")


def test_indexed_operands_without_rows_are_refused(ctx):
    """With an index the number of rows comes from the operand itself, which has to have some."""
    x, w, od, ix = _x(6, 64), _x(3, 32, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    for bad in (_x(6), torch.zeros(()), 3.0):
        _refused(lambda: ctx.grouped_linear(x, w, od, y_rows=ix, y=bad), "y is not a tensor")
        _refused(lambda: ctx.grouped_linear(x, w, od, y_rows=ix, residual=bad), "residual is not a tensor")
        _refused(lambda: ctx.grouped_linear_backward(bad, x, w, od, y_rows=ix), "dy is not a tensor")
        _refused(lambda: ctx.grouped_linear_backward(_x(6, 32), x, w, od, dx_rows=ix, dx=bad), "dx is not a tensor")


def test_backward_refusals(ctx):
    x, w, dy = _x(4, 64), _x(32, 64), _x(4, 32)
    back = ctx.linear_backward
    _refused(lambda: back(_x(4, 31), x, w), "dy has shape")
    _refused(lambda: back(dy.half(), x, w), "dy has type")
    _refused(lambda: back(dy, x, w, act="silu"), "z")
    _refused(lambda: back(dy, x, w, act="silu", z=_x(3, 32)), "z has shape")
    _refused(lambda: back(dy, x, w, act="silu", z=dy.float()), "z has type")
    _refused(lambda: back(dy, x, w, w_up=w, act="swiglu", z=dy), "z")
    _refused(lambda: back(dy, x, w, z_up=dy), "z_up")
    _refused(lambda: back(dy, x, w, need_dx=False, dx=x), "not needed")
    _refused(lambda: back(dy, x, w, db=_x(32, dtype=F)), "not needed")
    _refused(lambda: back(dy, x, w, accumulate=True), "accumulate")
    _refused(lambda: back(dy, x, w, accumulate=True, dw=w, need_db=True), "accumulate")


def test_backward_output_refusals(ctx, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(moe, "_raw_stream", lambda d: 0)
    x, w, dy = _x(4, 64), _x(32, 64), _x(4, 32)
    back = ctx.linear_backward
    _refused(lambda: back(dy, x, w, dx=_x(4, 63)), "dx has shape")
    _refused(lambda: back(dy, x, w, dw=_x(32, 63)), "dw has shape")
    _refused(lambda: back(dy, x, w, dw=_x(32, 64), dw_dtype=F), "dw_dtype")
    _refused(lambda: back(dy, x, w, dw_dtype=torch.int32), "dw_dtype")
    _refused(lambda: back(dy, x, w, need_db=True, db=_x(32)), "db has type")
    _refused(lambda: back(dy, x, w, w_up=w, act="swiglu", z=dy, z_up=dy, dw=_x(32, 64), dw_up=_x(32, 64, dtype=F)),
             "dw_up")


# ------------------------------------------------------------------ packed rows and launch plans
_HARNESS = r"""
#include "linear_tc.cuh"
#include <cstdio>
#include <cstdlib>
using namespace moe;
int main(int argc, char** argv) {
    const int slots[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
    int kind, E, rows, C, Q, out_n, f32, pair;
    while (std::scanf("%d %d %d %d %d %d %d %d", &kind, &E, &rows, &C, &Q, &out_n, &f32, &pair) == 8) {
        LinArgs a{};
        a.kind = kind; a.E = E; a.rows = rows; a.C = C; a.Q = Q; a.out_n = out_n;
        a.out_type = f32 ? LIN_F32 : LIN_BF16;
        a.a[0] = reinterpret_cast<void*>(1 << 20);
        a.b[0] = a.a[0];
        if (pair && kind == LIN_FWD) a.a[1] = reinterpret_cast<void*>((1 << 20) + (pair > 1 ? -4096 : 4096));
        if (pair && kind != LIN_FWD) a.b[1] = a.b[0];
        const LtPlan p = lt_plan(a, slots, 231424);
        std::printf("%d %d %d %d %d %d %d %d %d %d %d %d %d\n", p.bn, p.cg, p.split, p.ct, p.bbox, p.stages,
                    p.stage_bytes, p.off_ring, p.off_red, p.smem, p.n_ct, p.tmem_cols, p.grid);
    }
    // packed rows of groups never meet, and stay inside the copy
    std::srand(7);
    for (int i = 0; i < 2000; ++i) {
        const int E = 1 + std::rand() % 70;
        int at = std::rand() % 40, end = 0;
        for (int e = 0; e < E; ++e) {
            const int n = std::rand() % 3 ? std::rand() % 50 : 0;
            const int p = lin_packed(at, e);
            if (p % 16 || (n && p < end)) { std::printf("MEET\n"); return 1; }
            if (n) end = p + (n + 15) / 16 * 16;
            at += n;
        }
        if (end > lin_packed_rows(at, E)) { std::printf("OUTSIDE\n"); return 1; }
    }
    return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="no nvcc")
def test_plans_and_packed_rows(tmp_path):
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(_HARNESS)
    subprocess.run([NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    rng = random.Random(3)
    cases = [(0, 1, 1, 384, 5120, 0, 1, 0), (0, 1, 64, 2304, 5120, 0, 0, 1), (0, 1, 8192, 5120, 2304, 0, 0, 0),
             (0, 64, 12288, 2304, 5120, 0, 0, 1), (0, 1024, 48, 2304, 5120, 0, 0, 2), (1, 1, 8192, 5120, 2304, 0, 0, 1),
             (2, 64, 12288, 5120, 0, 2304, 0, 1), (2, 1, 2048, 5120, 0, 384, 1, 0), (0, 1, 1, 1, 1, 0, 0, 0),
             (2, 1, 1, 1, 0, 1, 0, 0), (1, 1, 1 << 20, 5120, 5120, 0, 1, 0)]
    for _ in range(400):
        cases.append((rng.randrange(3), rng.choice([1, 1, 2, 16, 64, 384, 1024]), rng.choice([1, 17, 300, 5000, 40000]),
                      rng.randint(1, 6000), rng.randint(1, 9000), rng.randint(1, 6000), rng.randrange(2),
                      rng.randrange(3)))
    out = subprocess.run([str(exe)], input="".join(" ".join(map(str, c)) + "\n" for c in cases), text=True,
                         capture_output=True, check=True).stdout.split("\n")
    slots = [0, 148, 74, 45, 33, 26, 22, 15, 15]
    for c, line in zip(cases, out):
        kind, E, rows, C, Q, out_n, f32, pair = c
        bn, cg, split, ct, bbox, stages, sb, ring, red, smem, n_ct, cols, grid = map(int, line.split())
        dual = kind == 0 and pair
        assert ct == (64 if dual else 128) and n_ct * ct * cg >= C > (n_ct - 1) * ct * cg, c
        assert bn in (16, 32, 64, 128, 256) and bn // cg >= (64 if kind == 2 else 16), c
        assert cg == 1 or split == 1, c
        assert 3 <= stages <= 12 and ring % 1024 == 0 and sb % 1024 == 0, c
        assert sb >= 16384 + bn // cg * 128 and red == ring + stages * sb, c
        assert ring >= 256 + 4 * (3 * E + 1) and smem <= 231424, c
        if split > 1:   # every item of four rows x 32 lanes has a place in the CTA that finishes it
            assert smem - 1024 - red >= -(-bn // (8 * split)) * 8 * split * 512, c
        assert bbox <= 256 and (bn // cg) % bbox == 0, c
        assert cols <= 512 and cols & (cols - 1) == 0 and cols >= 2 * bn, c
        assert grid >= 1 and grid % (cg * split) == 0 and grid <= slots[cg * split] * cg * split, c
    big, one = out[2].split(), out[0].split()
    assert (big[0], big[1]) == ("256", "2")            # large products run on CTA pairs
    assert one[0] == "16" and int(one[2]) > 1           # one token splits its sum over a cluster


# ------------------------------------------------------------------ formulas
@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "swiglu"])
def test_gradient_formulas_against_differences(name):
    g = torch.Generator().manual_seed(5)

    def rn(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    offs = [0, 3, 3, 7]
    x, w, wu = rn(7, 6), rn(3, 5, 6), rn(3, 5, 6) if name == "swiglu" else None
    b, bu = rn(3, 5), rn(3, 5) if name == "swiglu" else None
    dy = rn(7, 5)

    def loss():
        y, *_ = ref.forward(x, w, wu, b, bu, name, offs)
        return float((y * dy).sum())

    _, _, z, u, _, _ = ref.forward(x, w, wu, b, bu, name, offs)
    (dx, _), dw, db = ref.backward(dy, x, w, wu, z, u, name, offs, t16=torch.float64)
    pairs = [(x, dx), (w, dw[0][0]), (b, db[0][0])]
    if wu is not None:
        pairs += [(wu, dw[1][0]), (bu, db[1][0])]
    h = 1e-5
    for t, want in pairs:
        flat, got = t.view(-1), want.reshape(-1)
        for i in range(0, flat.numel(), 7):
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            # central differences: O(h^2) of a third derivative of order one, plus rounding / h
            assert abs((up - down) / (2 * h) - float(got[i])) < 1e-6 * max(1.0, abs(float(got[i])))
