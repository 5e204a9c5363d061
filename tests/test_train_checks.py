"""Refusals of the training operators, on the host: statuses of the C entry points (every check comes before any work),
the binding's own checks, and the header as strict C11."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from sub_bit_weight_b200 import build
    build.build()
    from sub_bit_weight_b200 import lib as binding
    return binding


def test_embedding_forward_arguments(lib):
    def call(ids=256, M=4, table=256, td=0, V=10, D=8, out=256, od=0):
        return lib._lib.lb_embedding_forward(vp(ids), M, vp(table), td, V, D, 1.0, vp(out), od, None)
    assert call(M=0, ids=0, table=0, out=0) == OK                 # nothing to do
    for bad in (dict(ids=0), dict(table=0), dict(out=0), dict(M=-1), dict(V=0), dict(D=0), dict(td=2), dict(od=-1),
                dict(ids=260), dict(table=258), dict(td=1, table=257), dict(out=257, od=1)):
        assert call(**bad) == INVALID, bad
    assert call(M=1 << 31) == UNSUPPORTED
    assert call(D=(1 << 25) + 1) == UNSUPPORTED


def test_embedding_backward_arguments(lib):
    need = lib.lb_embedding_backward_workspace_bytes(4, 10, 8)
    assert need > 0
    assert lib.lb_embedding_backward_workspace_bytes(-1, 10, 8) == 0
    assert lib.lb_embedding_backward_workspace_bytes(4, 0, 8) == 0

    def call(ids=256, M=4, dout=256, dd=0, V=10, D=8, out=256, od=0, ws=256, wb=need):
        return lib._lib.lb_embedding_backward(vp(ids), M, vp(dout), dd, V, D, 1.0, vp(out), od, vp(ws), wb, None)
    for bad in (dict(ids=0), dict(dout=0), dict(out=0), dict(ws=0), dict(M=-1), dict(V=0), dict(D=0), dict(dd=7),
                dict(od=2), dict(ids=252), dict(dout=258), dict(out=258), dict(ws=128), dict(wb=need - 1)):
        assert call(**bad) == INVALID, bad
    assert call(M=1 << 31) == UNSUPPORTED


def test_cross_entropy_arguments(lib):
    f, g = lib._lib.lb_cross_entropy_forward, lib._lib.lb_cross_entropy_gradient
    need = lib.lb_cross_entropy_forward_workspace_bytes(200, 64, 1000)
    grad = lib.lb_cross_entropy_gradient_workspace_bytes(200, 64, 1000)
    assert grad > need > 0
    # the scratch follows the rows taken at a time, not M
    assert lib.lb_cross_entropy_gradient_workspace_bytes(100000, 64, 1000, rows=128) < 2 ** 20 + 2 * 128 * 1000 * 2 + 1000 * 64 * 4

    def fwd(H=256, W=256, lab=256, M=200, D=64, V=1000, loss=256, lse=256, ws=256, wb=need):
        return f(vp(H), vp(W), vp(lab), M, D, V, vp(loss), vp(lse), vp(ws), wb, None)

    def bwd(H=256, W=256, lab=256, w=256, M=200, D=64, V=1000, rows=0, loss=256, dH=256, dW=256, ws=256, wb=grad):
        return g(vp(H), vp(W), vp(lab), vp(w), M, D, V, rows, vp(loss), vp(dH), vp(dW), vp(ws), wb, None)
    assert fwd(M=0, H=0) == OK and bwd(M=0, H=0, dW=0) == OK
    for call, more in ((fwd, [dict(lse=0), dict(lse=258)]), (bwd, [dict(w=0), dict(dH=0), dict(w=258), dict(dH=264),
                                                                    dict(dW=264), dict(rows=-1)])):
        for bad in [dict(H=0), dict(W=0), dict(lab=0), dict(loss=0), dict(ws=0), dict(M=-1), dict(D=0), dict(V=0),
                    dict(H=264), dict(W=264), dict(lab=260), dict(ws=192), dict(wb=100)] + more:
            assert call(**bad) == INVALID, bad
        assert call(D=60) == UNSUPPORTED                          # rows that are not a multiple of 16 bytes
        assert call(V=(1 << 28) + 1) == UNSUPPORTED


def test_orthogonalise_arguments(lib):
    i = ctypes.c_int
    f = lib._lib.lb_orthogonalise
    need = lib.lb_orthogonalise_workspace_bytes([(300, 100)])
    assert need > 300 * 100 * 4
    assert lib.lb_orthogonalise_workspace_bytes([]) == 0
    assert lib.lb_orthogonalise_workspace_bytes([(0, 4)]) == 0
    assert lib.lb_orthogonalise_workspace_bytes([(512, 16)] * 4) == 0                     # done without scratch
    assert lib.lb_orthogonalise_workspace_bytes([(300, 100)], torch.bfloat16) < need      # no low halves

    def call(G=256, dt=0, r=300, c=100, n=1, steps=5, eps=1e-7, O=256, ws=256, wb=need):
        return f((vp * 1)(vp(G)), dt, (i * 1)(r), (i * 1)(c), n, steps, eps, (vp * 1)(vp(O)), vp(ws), wb, None)
    assert call(n=0) == OK
    for bad in (dict(G=0), dict(O=0), dict(ws=0), dict(r=0), dict(c=-3), dict(n=-1), dict(dt=2), dict(steps=0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(G=258), dict(O=257), dict(ws=100), dict(wb=need - 1)):
        assert call(**bad) == INVALID, bad
    assert call(steps=11) == UNSUPPORTED
    assert call(r=2049, c=2049, wb=1 << 40) == UNSUPPORTED
    assert f(None, 0, None, None, 1, 5, 1e-7, None, None, 0, None) == INVALID


def test_binding_refuses(lib):
    ids, table = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    bf = torch.bfloat16
    with pytest.raises(TypeError, match="ids must be a CUDA"):
        lib.lb_embedding_forward(ids, table)
    with pytest.raises(ValueError, match="table must be"):
        lib.lb_embedding_forward(ids, table[0])
    with pytest.raises(ValueError, match="dout must be"):
        lib.lb_embedding_backward(ids, torch.zeros(4, 8), 5)
    with pytest.raises(TypeError, match="CUDA"):
        lib.lb_embedding_backward(ids, torch.zeros(3, 8), 5)
    H, W = torch.zeros(3, 8, dtype=bf), torch.zeros(5, 8, dtype=bf)
    for call in (lambda **k: lib.lb_cross_entropy_forward(**k),
                 lambda **k: lib.lb_cross_entropy_gradient(weight=torch.zeros(3), **k)):
        with pytest.raises(ValueError, match="H must be"):
            call(H=H, W=W[:, :4], labels=ids)
        with pytest.raises(ValueError, match="labels must hold 3"):
            call(H=H, W=W, labels=ids[:2])
        with pytest.raises(TypeError, match="H must be a CUDA"):
            call(H=H, W=W, labels=ids)
    with pytest.raises(ValueError, match="weight must hold 3"):
        lib.lb_cross_entropy_gradient(H, W, ids, torch.zeros(2))
    assert lib.lb_orthogonalise([]) == []
    for bad in ([torch.zeros(3)], [torch.zeros(3, 4), torch.zeros(0, 4)], [None]):
        with pytest.raises(ValueError, match=rf"G\[{len(bad) - 1}\] must be a matrix"):
            lib.lb_orthogonalise(bad)
    with pytest.raises(TypeError, match="G must be float32 or bfloat16"):
        lib.lb_orthogonalise([torch.zeros(3, 4, dtype=torch.float16)])
    with pytest.raises(TypeError, match=r"G\[0\] must be a CUDA"):
        lib.lb_orthogonalise([torch.zeros(3, 4)])


def test_binding_refuses_sizes_past_a_c_int(lib):
    """ctypes would cut them to 32 bits: a matrix of 2^32 + 16 rows would be taken for one of 16."""
    huge = (1 << 32) + 16
    wide = lambda n, m, dtype=torch.float32: torch.zeros(1, 1, dtype=dtype).expand(n, m)   # no memory behind it
    ids, bf = torch.zeros(3, dtype=torch.int64), torch.bfloat16
    with pytest.raises(ValueError, match="V must be"):
        lib.lb_embedding_forward(ids, wide(huge, 8))
    with pytest.raises(ValueError, match="V must be"):
        lib.lb_embedding_backward(ids, torch.zeros(3, 8), huge)
    with pytest.raises(ValueError, match="V must be"):
        lib.lb_embedding_backward(ids, torch.zeros(3, 8), -1)
    with pytest.raises(ValueError, match="V must be"):
        lib.lb_cross_entropy_forward(wide(3, 8, bf), wide(huge, 8, bf), ids)
    with pytest.raises(ValueError, match="M must be"):
        lib.lb_cross_entropy_forward(wide(huge, 8, bf), wide(5, 8, bf), ids[:1].expand(huge))
    with pytest.raises(ValueError, match="rows must be"):
        lib.lb_cross_entropy_gradient(wide(3, 8, bf), wide(5, 8, bf), ids, torch.zeros(3), rows=huge)
    with pytest.raises(ValueError, match=r"G\[1\] has a side"):
        lib.lb_orthogonalise([torch.zeros(3, 4), wide(huge, 16)])


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(lib):
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    table = torch.zeros(5, 8, device="cuda")
    with pytest.raises(TypeError, match="ids must be torch.int64"):
        lib.lb_embedding_forward(ids.int(), table)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        lib.lb_embedding_forward(ids, table.half())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        lib.lb_embedding_forward(ids, table, dtype=torch.float16)
    with pytest.raises(ValueError, match="table must be contiguous"):
        lib.lb_embedding_forward(ids, table[:, :4])
    with pytest.raises(ValueError, match="workspace must hold"):
        lib.lb_embedding_backward(ids, table[:3], 5, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="workspace is on cpu"):
        lib.lb_embedding_backward(ids, table[:3], 5, workspace=torch.empty(4096, dtype=torch.uint8))
    H, W = torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError, match="W must be torch.bfloat16"):
        lib.lb_cross_entropy_forward(H, W.float(), ids)
    with pytest.raises(TypeError, match="labels must be a CUDA"):
        lib.lb_cross_entropy_forward(H, W, ids.cpu())
    with pytest.raises(lib.LittleBitError, match="UNSUPPORTED"):
        lib.lb_cross_entropy_forward(H[:, :4].contiguous(), W[:, :4].contiguous(), ids)
    with pytest.raises(TypeError, match=r"G\[1\] must be torch.float32"):
        lib.lb_orthogonalise([table, table.bfloat16()])
    with pytest.raises(lib.LittleBitError, match="UNSUPPORTED"):
        lib.lb_orthogonalise([table], steps=11)
    with pytest.raises(lib.LittleBitError, match="INVALID"):
        lib.lb_orthogonalise([table], steps=0)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_from_c(lib, tmp_path):
    src = tmp_path / "train.c"
    src.write_text("""
#include "littlebit_train.h"
#include <stdio.h>
int main(void)
{
    const int rows[1] = {300}, cols[1] = {100};
    if (lb_cross_entropy_forward(NULL, NULL, NULL, 1, 8, 8, NULL, NULL, NULL, 0, NULL) != LB_ERR_INVALID_ARG) return 1;
    if (lb_embedding_forward(NULL, 0, NULL, LB_BF16, 4, 4, 1.0f, NULL, LB_F32, NULL) != LB_OK) return 2;
    if (lb_orthogonalise_workspace_bytes(rows, cols, 1, LB_F32) == 0) return 3;
    if (lb_cross_entropy_gradient_workspace_bytes(4, 8, 8, 1, 0) % 256 != 0) return 4;
    puts("OK");
    return 0;
}
""")
    exe = tmp_path / "train"
    libdir = os.path.dirname(lib.LIB_PATH)
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                        str(src), "-o", str(exe), "-L", libdir, "-llittlebit", "-Wl,-rpath," + libdir],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "OK", (r.returncode, r.stdout, r.stderr)


def test_workspace_sizes_of_refused_shapes(lib):
    """A size that the call refuses has no scratch: the query answers 0, at once."""
    f32, bf = torch.float32, torch.bfloat16
    for dtype in (f32, bf):
        for bad in ((2049, 2049), (300000, 300000), (2 ** 31 - 1, 2 ** 31 - 1), ((1 << 24) + 1, 4), (4, (1 << 24) + 1)):
            assert lib.lb_orthogonalise_workspace_bytes([(300, 100), bad], dtype) == 0, bad
        assert lib.lb_orthogonalise_workspace_bytes([(2048, 2048), (1 << 24, 100)], dtype) > 0
    assert lib.lb_embedding_backward_workspace_bytes(4, 10, 1 << 23) > 0
    assert lib.lb_embedding_backward_workspace_bytes(4, 10, (1 << 23) + 1) == 0
    assert lib.lb_embedding_backward_workspace_bytes(1 << 31, 10, 8) == 0
    for query in (lib.lb_cross_entropy_forward_workspace_bytes, lib.lb_cross_entropy_gradient_workspace_bytes):
        assert query(4, 64, 100) > 0
        for bad in ((4, 60, 100), (-1, 64, 100), (4, (1 << 20) + 8, 100), (4, 64, (1 << 28) + 1), ((1 << 28) + 1, 64, 100)):
            assert query(*bad) == 0, bad


@pytest.mark.gpu
def test_refused_ranks_take_no_scratch(lib):
    G = torch.zeros(3000, 2500, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(lib.LittleBitError, match="UNSUPPORTED"):
        lib.lb_orthogonalise([G])
    assert torch.cuda.max_memory_allocated() - before <= G.numel() * 2 + 4096         # the output alone


def test_workspace_sizes_refuse_past_a_c_int(lib):
    """A number that ctypes would cut to 32 bits, in every argument of the size functions, and of the call's own steps."""
    huge = (1 << 32) + 4
    for k in range(1, 3):
        args = [4, 10, 8]
        args[k] = huge
        with pytest.raises(ValueError, match="fit"):
            lib.lb_embedding_backward_workspace_bytes(*args)
    assert lib.lb_embedding_backward_workspace_bytes((1 << 64) + 4, 10, 8) == 0
    for query, n in ((lib.lb_cross_entropy_forward_workspace_bytes, 3), (lib.lb_cross_entropy_gradient_workspace_bytes, 5)):
        for k in range(n):
            args = [4, 8, 10, True, 0][:n]
            if k == 3:
                continue
            args[k] = huge
            with pytest.raises(ValueError, match="fit"):
                query(*args)
    for bad in ((huge, 16), (16, huge)):
        with pytest.raises(ValueError, match="fit"):
            lib.lb_orthogonalise_workspace_bytes([(16, 16), bad])
    with pytest.raises(ValueError, match="steps must fit"):
        lib.lb_orthogonalise([torch.zeros(3, 4)], steps=(1 << 32) + 5)


@pytest.mark.gpu
def test_no_workspace_where_none_is_needed(lib):
    i = ctypes.c_int
    G = torch.randn(512, 16, device="cuda")
    O = torch.empty(512, 16, dtype=torch.bfloat16, device="cuda")
    assert lib.lb_orthogonalise_workspace_bytes([(512, 16)]) == 0
    st = lib._lib.lb_orthogonalise((vp * 1)(G.data_ptr()), 0, (i * 1)(512), (i * 1)(16), 1, 5, 1e-7, (vp * 1)(O.data_ptr()),
                                   None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == OK and torch.equal(O, lib.lb_orthogonalise([G])[0])
