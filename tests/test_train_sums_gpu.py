"""Long sums on the tensor cores, whose accumulators truncate, against 64-bit values: sums of one sign that a later term
all but cancels, and updates whose small singular values an error of the Gram matrix would move."""

import pytest
import torch

from test_train_gpu import BF16, MMA, _gen, _off, _orth_ref, _within, lib  # noqa: F401

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


# The gradients of the loss where every probability is a power of two (all logits zero), so that G is known to the last bit.
# Weights of 1 and 255/256 give products finer than the accumulator; nearly all terms have one sign, and the last ones (the
# label's) cancel the sum, so that a bias of the sum shows beside the rounding of the small result.  Bound: 64 additions of
# 2^-22 for each 1024 k of the magnitudes there, 2^-24 of the largest sum for each of these pieces added, the rounding.

def _weights(M):
    return torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, 255 / 256)


def test_cross_entropy_gradient_of_hidden_states_over_a_long_vocabulary(lib):  # noqa: F811
    M, D, V = 512, 9472, 1 << 17                                  # 74 tiles: the vocabulary is not cut
    g = _gen(1)
    W = torch.empty(V, D, dtype=BF16, device="cuda")
    for v in range(0, V, 1 << 14):
        W[v:v + (1 << 14)] = 1 + torch.randint(0, 128, (1 << 14, D), generator=g, device="cuda") / 128
    W[V - 1] = 1.5
    H = torch.zeros(M, D, dtype=BF16, device="cuda")
    labels = torch.full((M,), V - 1, device="cuda")
    weight = _weights(M)
    _, dH, _ = lib.lb_cross_entropy_gradient(H, W, labels, weight, head=False)
    p = weight.double()[:, None] / V
    at_label = (weight.double() * (1 / V - 1)).to(BF16).double()[:, None]
    sums = torch.zeros(D, dtype=torch.float64, device="cuda")
    for v in range(0, V - 1, 1 << 14):
        sums += W[v:min(v + (1 << 14), V - 1)].sum(0, dtype=torch.float64)
    ref = p * sums + at_label * 1.5
    pieces = V // 1024
    bound = 64 * MMA * (p * sums + 1.5) + pieces * 2.0 ** -24 * 2.0
    assert float(ref.abs().max()) < 0.02                          # the sum is all but cancelled
    _within(dH, ref, bound + 2.0 ** -8 * (ref.abs() + bound))


def test_cross_entropy_gradient_of_the_vocabulary_over_many_rows(lib):  # noqa: F811
    M, D, V = 32768, 256, 256
    g = _gen(2)
    H = (1.5 + torch.randint(-2, 3, (M, D), generator=g, device="cuda") / 128).to(BF16)
    W = torch.zeros(V, D, dtype=BF16, device="cuda")
    labels = torch.arange(M, device="cuda") // 128
    weight = _weights(M)
    _, _, dW = lib.lb_cross_entropy_gradient(H, W, labels, weight, rows=M)
    G = (weight.double() / V)[:, None].expand(M, V).clone()
    G[torch.arange(M, device="cuda"), labels] = (weight.double() * (1 / V - 1)).to(BF16).double()
    Hd = H.double()
    ref = G.T @ Hd
    mags = torch.stack([G[m:m + 1024].T.abs() @ Hd[m:m + 1024] for m in range(0, M, 1024)])
    bound = 64 * MMA * mags.sum(0) + len(mags) * 2.0 ** -24 * 200.0
    _within(dW, ref, bound + 2.0 ** -8 * (ref.abs() + bound))


@pytest.mark.parametrize("M,D,rows", [(300, 264, 0), (5, 1032, 0), (700, 520, 256), (2, 8, 0)])
def test_cross_entropy_gradient_of_hidden_states_keeps_the_label_entry(lib, M, D, rows):  # noqa: F811
    """p - 1 = -511/512 lies halfway between two bfloat16 numbers; rounded, it would scale each row's part of W[label] by
    2^-9 of it, the same way in every column.  All else is exact (p = 2^-9), so the result is within the accumulation's
    errors of half a step of itself: 64 additions of 2^-22 of the magnitudes, and a float32 rounding or two."""
    V = 512
    g = _gen(M)
    W = torch.randn(V, D, generator=g, device="cuda").to(BF16)
    H = torch.zeros(M, D, dtype=BF16, device="cuda")
    labels = torch.randint(0, V, (M,), generator=g, device="cuda")
    labels[1::3] = -100
    weight = torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, 0.25)
    _, dH, _ = lib.lb_cross_entropy_gradient(H, W, labels, weight, rows=rows)
    ok = (labels >= 0)[:, None]
    Wd = W.double()
    w = weight.double()[:, None] * ok
    ref = w * (Wd.sum(0) / V - Wd[labels.clamp(min=0)])
    e = w * 65 * MMA * (Wd.abs().sum(0) / V + Wd[labels.clamp(min=0)].abs())
    half_step = torch.exp2(torch.floor(torch.log2((ref.abs() + e).clamp(min=1e-30))) - 8)
    _within(dH, ref, torch.where(ok, e + half_step, 0.0))
