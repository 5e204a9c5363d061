"""Training operators past the limits at which a call is cut into sets: matrices, shapes and vocabulary rows."""

import pytest
import torch

from test_train_gpu import BF16, F32, SMOOTH, _gen, _off, _orth_ref, lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalise_more_small_matrices_than_one_set(lib, dtype):  # noqa: F811
    """130 matrices that a block does whole: two full sets of 64 and a rest."""
    g = _gen(1)
    shapes = [(40 + 3 * i, 1 + i % 20) if i % 3 else (1 + i % 20, 40 + 3 * i) for i in range(130)]
    G = [torch.randn(s, generator=g, device="cuda").to(dtype) for s in shapes]
    for i, (X, O) in enumerate(zip(G, lib.lb_orthogonalise(G))):
        assert _off(O, _orth_ref(X)) <= SMOOTH, (i, shapes[i])


@pytest.mark.parametrize("shape", [(700, 40), (300, 70), (70, 300), (400, 130)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalise_more_equal_matrices_than_one_set(lib, shape, dtype):  # noqa: F811
    """A shape whose matrices go on in the next set, with another before and after it, for each way of the n x n part."""
    g = _gen(2)
    shapes = [(1500, 600)] + [shape] * 66 + [(900, 33)]
    G = [torch.randn(s, generator=g, device="cuda").to(dtype) for s in shapes]
    for i, (X, O) in enumerate(zip(G, lib.lb_orthogonalise(G))):
        assert _off(O, _orth_ref(X)) <= SMOOTH, (i, shapes[i])
    assert lib.lb_train_status() == lib.LB_OK


@pytest.mark.parametrize("D", [8, 9])
def test_embedding_backward_more_rows_than_a_block_flags_at_once(lib, D):  # noqa: F811
    """A block keeps flags of 4096 rows at a time: ids on both sides of each such boundary and at the ends of every block's
    rows, each once, so that the result is known to the last bit; the output held NaN before."""
    V = 1_300_001
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    per = -(-V // blocks)
    assert per > 2 * 4096
    near = [0, 1, 4094, 4095, 4096, 4097, 8191, 8192, 8193, per - 2, per - 1]
    ids = sorted({b * per + n for b in range(blocks) for n in near} & set(range(V)) | {V - 1})
    g = _gen(3)
    ids = torch.tensor(ids, device="cuda")
    ids = ids[torch.randperm(ids.numel(), generator=g, device="cuda")]
    M = ids.numel()
    dout = torch.randn(M, D, generator=g, device="cuda")
    dtable = torch.full((V, D), float("nan"), device="cuda")
    need = lib.lb_embedding_backward_workspace_bytes(M, V, D)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = lib._lib.lb_embedding_backward(ids.data_ptr(), M, dout.data_ptr(), lib.LB_F32, V, D, 1.0, dtable.data_ptr(),
                                        lib.LB_F32, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == lib.LB_OK
    ref = torch.zeros(V, D, device="cuda")
    ref[ids] = dout
    assert torch.equal(dtable, ref)
