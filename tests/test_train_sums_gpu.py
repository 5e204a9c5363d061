"""Long sums on the tensor cores, whose accumulators truncate, against 64-bit values: sums of one sign that a later term
all but cancels, and updates whose small singular values an error of the Gram matrix would move."""

import pytest
import torch

from test_train_gpu import BF16, _gen, _off, _orth_ref, lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _spectrum(g, m, n, kind):
    """A matrix with singular values that fall off, or of which one dominates."""
    U, _ = torch.linalg.qr(torch.randn(m, n, generator=g, device="cuda", dtype=torch.float64))
    V, _ = torch.linalg.qr(torch.randn(n, n, generator=g, device="cuda", dtype=torch.float64))
    j = torch.arange(1, n + 1, device="cuda", dtype=torch.float64)
    s = {"1/j2": 1 / j ** 2, "spike": torch.where(j == 1, 1.0, 0.002)}[kind]
    return ((U * s) @ V.T).float()


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("kind", ["1/j2", "spike"])
def test_orthogonalise_long_matrices_of_hard_spectra_in_a_large_set(lib, kind, dtype):  # noqa: F811
    """11008 x 800 among as many matrices as a block of layers has, so that no matrix needs its long axis cut to occupy the
    GPU; and by itself, where it is cut.  What bfloat16's rounding alone makes of a result whose mantissas are spread
    evenly is 1.5e-3 of its norm (2^-7 / sqrt(12) over the root mean square 1.53 of a mantissa), a little more for a
    normal distribution; 2.2e-3 leaves the Gram matrix's errors 1.4e-3."""
    g = _gen(5)
    hard = _spectrum(g, 11008, 800, kind).to(dtype)
    ref = _orth_ref(hard)
    G = [hard] + [torch.randn(11008, 800, generator=g, device="cuda") for _ in range(5)] \
        + [torch.randn(4096, 800, generator=g, device="cuda") for _ in range(6)] \
        + [torch.randn(4096, 544, generator=g, device="cuda") for _ in range(16)]
    assert _off(lib.lb_orthogonalise([X.to(dtype) for X in G])[0], ref) <= 2.2e-3
    assert _off(lib.lb_orthogonalise([hard])[0], ref) <= 2.2e-3


@pytest.mark.parametrize("kind", ["1/j2", "spike"])
def test_orthogonalise_hard_spectra_of_the_largest_rank(lib, kind):  # noqa: F811
    """The n x n products are longest at rank 2048."""
    hard = _spectrum(_gen(6), 2200, 2048, kind)
    assert _off(lib.lb_orthogonalise([hard])[0], _orth_ref(hard)) <= 2.2e-3
