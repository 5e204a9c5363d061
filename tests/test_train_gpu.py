"""The operators around the layers in a training step against plain 64-bit forms, on the GPU.

Tolerances are bounds, not observations.  A rounding moves a value by at most half a step: 2^-8 of it for bfloat16,
2^-11 for binary16, 2^-24 for float32.  The tensor cores add 16 products at a time to a float32 accumulator with
truncation; four units of the accumulator's last place per addition (2^-22 of the sum of magnitudes) bounds that
generously.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
MMA = 2.0 ** -22


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from sub_bit_weight_b200 import lib as _lib
    return _lib


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _within(out, ref, bound, what=""):
    err = (out.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / bound.clamp(min=1e-300)).max()))


# ---------------------------------------------------------------------------------------------- embedding

def _ids(g, shape, V):
    n = int(np.prod(shape))
    u = torch.rand(n, generator=g, device="cuda") ** 3            # a few frequent ids, a long tail
    return (u * (V + 2)).long().sub_(1).reshape(shape)            # -1 and V among them


@pytest.mark.parametrize("shape,V,D,scale", [
    ((1,), 5, 3, 1.0), ((3, 7), 11, 8, 1.0), ((65,), 100, 33, 11.5), ((2, 500), 1000, 1028, 64.0),
    ((4096,), 32000, 256, 1.0), ((5,), 3, 8192 + 4, -2.5),
])
@pytest.mark.parametrize("src", [F32, BF16])
@pytest.mark.parametrize("dst", [F32, BF16])
def test_embedding_forward(lib, shape, V, D, scale, src, dst):
    g = _gen(V + D)
    ids = _ids(g, shape, V)
    table = torch.randn(V, D, generator=g, device="cuda").to(src)
    out = lib.lb_embedding_forward(ids, table, scale=scale, dtype=dst)
    ok = (ids >= 0) & (ids < V)
    rows = table[torch.where(ok, ids, 0)].float() * torch.tensor(scale, dtype=F32, device="cuda")
    ref = torch.where(ok[..., None], rows, 0.0).to(dst)           # one product in float32, one rounding: the same bits
    assert out.shape == (*shape, D) and torch.equal(out, ref)


def test_embedding_forward_far_rows_and_foreign_ids(lib):
    V, D = 540_000, 4096                                           # 2.2e9 elements: offsets beyond 32 bits
    table = torch.zeros(V, D, dtype=BF16, device="cuda")
    table[V - 1] = 3.0
    table[0] = 5.0
    ids = torch.tensor([V - 1, -1, V, 2 ** 62, -2 ** 62, 0], device="cuda")
    out = lib.lb_embedding_forward(ids, table)
    assert torch.equal(out[:, 0].float().cpu(), torch.tensor([3.0, 0, 0, 0, 0, 5.0]))
    assert torch.equal(out[:, 0], out[:, -1])
    d = torch.ones(6, D, dtype=BF16, device="cuda")
    grad = lib.lb_embedding_backward(ids, d, V, dtype=BF16)
    assert float(grad[V - 1].sum()) == D and float(grad[0].sum()) == D and int(torch.count_nonzero(grad)) == 2 * D


@pytest.mark.parametrize("M,V,D", [
    (1, 1, 1), (1, 40, 5), (31, 7, 33), (257, 3, 64), (1000, 5000, 130), (4096, 50, 72), (4097, 900, 48),
    (16384, 257, 24), (16385, 300, 16), (40000, 5, 12), (70001, 20000, 40),
])
@pytest.mark.parametrize("src,dst", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
def test_embedding_backward(lib, M, V, D, src, dst):
    g = _gen(M + V)
    ids = _ids(g, (M,), V)
    dout = torch.randn(M, D, generator=g, device="cuda").to(src)
    scale = 1.75
    out = lib.lb_embedding_backward(ids, dout, V, scale=scale, dtype=dst)
    ok = (ids >= 0) & (ids < V)
    at = torch.where(ok, ids, V)
    ref, mag = (torch.zeros(V + 1, D, dtype=torch.float64, device="cuda").index_add_(0, at, x)[:V] * scale
                for x in (dout.double(), dout.double().abs()))
    n = torch.bincount(at, minlength=V + 1)[:V, None].double()
    # n - 1 additions of 2^-24 each, the product with the scale, the rounding of the result
    _within(out, ref, (n * 2.0 ** -24 + 2.0 ** -24) * mag + HALF_STEP[dst] * ref.abs())
    assert not out[n[:, 0] == 0].any()
    assert torch.equal(out, lib.lb_embedding_backward(ids, dout, V, scale=scale, dtype=dst))   # the same bits every time


@pytest.mark.parametrize("M", [0, 9])
def test_embedding_backward_overwrites_everything(lib, M):
    V, D = 9000, 20
    dtable = torch.full((V, D), float("nan"), device="cuda")
    ids = torch.full((M,), -1, dtype=torch.int64, device="cuda")
    dout = torch.full((M, D), float("inf"), device="cuda")        # no token: never read into a sum
    ws = torch.empty(lib.lb_embedding_backward_workspace_bytes(M, V, D) + 1, dtype=torch.uint8, device="cuda")
    st = lib._lib.lb_embedding_backward(ids.data_ptr(), M, dout.data_ptr(), lib.LB_F32, V, D, 1.0, dtable.data_ptr(),
                                        lib.LB_F32, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == lib.LB_OK and not dtable.any()


def test_embedding_unaligned_rows(lib):
    """Arrays that start one element past a 16-byte boundary, and a NaN that stays in its token's row."""
    V, D, M = 50, 16, 300
    g = _gen(3)
    flat = torch.randn(V * D + 1, generator=g, device="cuda")
    table = flat[1:].view(V, D)
    ids = _ids(g, (M,), V)
    ok = (ids >= 0) & (ids < V)
    out = lib.lb_embedding_forward(ids, table)
    assert torch.equal(out, torch.where(ok[:, None], table[torch.where(ok, ids, 0)], 0.0))
    dflat = torch.randn(M * D + 1, generator=g, device="cuda").to(BF16)
    dout = dflat[1:].view(M, D)
    j = int(torch.nonzero(ok)[0, 0])
    dout[j, 3] = float("nan")
    grad = lib.lb_embedding_backward(ids, dout, V)
    nan = torch.isnan(grad)
    assert int(nan.sum()) == 1 and bool(nan[ids[j], 3])


# ---------------------------------------------------------------------------------------------- loss

def _loss_inputs(seed, M, D, V, sure=3.0, wscale=0.05):
    g = _gen(seed)
    W = (torch.randn(V, D, generator=g, device="cuda") * wscale).to(BF16)
    labels = torch.randint(0, V, (M,), generator=g, device="cuda")
    H = torch.randn(M, D, generator=g, device="cuda")
    w = W[labels].float()
    H += sure * torch.rand(M, 1, generator=g, device="cuda") * w / w.norm(dim=1, keepdim=True).clamp(min=1e-6)
    skip = torch.rand(M, generator=g, device="cuda") < 0.2
    labels[skip] = torch.tensor([-100, V, -1, 2 ** 40], device="cuda")[torch.arange(int(skip.sum()), device="cuda") % 4]
    return H.to(BF16), W, labels


def _loss_ref(H, W, labels):
    H, W = H.double(), W.double()
    z = H @ W.T
    ok = (labels >= 0) & (labels < W.shape[0])
    at = torch.where(ok, labels, 0)[:, None]
    lse = torch.logsumexp(z, 1)
    loss = torch.where(ok, lse - z.gather(1, at)[:, 0], 0.0)
    mag = H.abs() @ W.abs().T                                     # sum of magnitudes behind each logit
    return z, lse, loss, ok, at, mag


def _logit_bound(D, mag):
    # 1024 k are at most 64 additions of 16; the chunks are added in float32; then 2^-23 for the change of base
    return (64 + D / 1024 + 2) * MMA * mag + 2.0 ** -22 * mag


def _lse_bound(D, mag, z, lse):
    # the logits' errors, weighted by the softmax; 2^-22 for each exponential, 2^-24 per addition over at most 64 in a
    # row of a thread and the merges after it; log and the product with ln 2: 2^-22 of the result
    p = torch.exp(z - lse[:, None])
    return (p * _logit_bound(D, mag)).sum(1) + 2.0 ** -17 + 2.0 ** -21 * lse.abs()


LOSS_SIZES = [(1, 8, 1), (1, 64, 1000), (3, 16, 129), (16, 520, 5003), (64, 1088, 300), (65, 128, 256), (128, 72, 4100),
              (129, 256, 1025), (300, 264, 1111), (513, 2056, 777)]


@pytest.mark.parametrize("M,D,V", LOSS_SIZES)
def test_cross_entropy_forward(lib, M, D, V):
    H, W, labels = _loss_inputs(M + D + V, M, D, V)
    loss, lse = lib.lb_cross_entropy_forward(H, W, labels)
    z, lse_r, loss_r, ok, at, mag = _loss_ref(H, W, labels)
    b = _lse_bound(D, mag, z, lse_r)
    _within(lse, lse_r, b)
    _within(loss, loss_r, torch.where(ok, b + _logit_bound(D, mag).gather(1, at)[:, 0] + 2.0 ** -23 * loss_r, 0.0))
    assert lib.lb_train_status() == lib.LB_OK


@pytest.mark.parametrize("M", [5, 200])
def test_cross_entropy_large_logits(lib, M):
    """Logits of several hundred, in the last vocabulary tile as well as the first: no overflow, no lost maximum."""
    D, V = 128, 700
    H, W, labels = _loss_inputs(M, M, D, V, sure=0.0, wscale=4.0)
    W[V - 1] = (H[0].float().sign() * 8.0).to(BF16)
    W[0] = (-H[0].float().sign() * 8.0).to(BF16)
    loss, lse = lib.lb_cross_entropy_forward(H, W, labels)
    z, lse_r, loss_r, ok, at, mag = _loss_ref(H, W, labels)
    assert float(z.abs().max()) > 500
    b = _lse_bound(D, mag, z, lse_r)
    _within(lse, lse_r, b)
    _within(loss, loss_r, torch.where(ok, b + _logit_bound(D, mag).gather(1, at)[:, 0] + 2.0 ** -23 * loss_r, 0.0))


def _grad_bounds(H, W, labels, weight, D):
    z, lse, loss, ok, at, mag = _loss_ref(H, W, labels)
    p = torch.exp(z - lse[:, None])
    w = torch.where(ok, weight.double(), 0.0)[:, None]
    G = p.clone()
    G.scatter_add_(1, at, -torch.ones_like(lse)[:, None])
    G = torch.where(ok[:, None], G, 0.0) * w
    # relative error of an entry: the logit's and lse's errors, e in binary16, G in bfloat16, the weight's quotient; an
    # entry far below its tile's maximum is held to 2^-39 of it
    dz = _logit_bound(D, mag) + _lse_bound(D, mag, z, lse)[:, None]
    eG = (p * w.abs()) * (dz + 2.0 ** -11 + 2.0 ** -20) + G.abs() * (2.0 ** -8 + 2.0 ** -22) + w.abs() * 2.0 ** -38
    eG = torch.where(ok[:, None], eG, 0.0)
    return G, eG, loss


GRAD_SIZES = [(1, 8, 3, 0), (1, 64, 1000, 0), (5, 16, 257, 0), (300, 264, 1111, 0), (300, 264, 1111, 100),
              (700, 520, 2050, 0), (257, 1032, 515, 256), (130, 64, 20000, 0)]


@pytest.mark.parametrize("M,D,V,rows", GRAD_SIZES)
@pytest.mark.parametrize("head", [True, False])
@pytest.mark.parametrize("uniform", [True, False])
def test_cross_entropy_gradient(lib, M, D, V, rows, head, uniform):
    H, W, labels = _loss_inputs(M + V, M, D, V)
    g = _gen(M * 3 + 1)
    weight = (torch.full((M,), 1.0 / M, device="cuda") if uniform
              else torch.randn(M, generator=g, device="cuda") * 2.0 / M)
    loss, dH, dW = lib.lb_cross_entropy_gradient(H, W, labels, weight, head=head, rows=rows)
    G, eG, loss_r = _grad_bounds(H, W, labels, weight, D)
    Hd, Wd = H.double(), W.double()

    def check(out, A, eA, B, K, what):
        ref, mag = A @ B, A.abs() @ B.abs()
        # errors of G, the sum over K in steps of 16, pieces and ranges in float32, the scale, the rounding
        bound = eA @ B.abs() + ((K / 16 + 2) * MMA + 20 * 2.0 ** -24) * mag
        _within(out, ref, bound + 2.0 ** -8 * (ref.abs() + bound) + 1e-38, what)

    check(dH, G, eG, Wd, V, "dH")
    if head:
        check(dW, G.T, eG.T, Hd, M, "dW")
    else:
        assert dW is None
    z, lse, _, ok, at, mag = _loss_ref(H, W, labels)
    _within(loss, loss_r, torch.where(ok, _lse_bound(D, mag, z, lse) + _logit_bound(D, mag).gather(1, at)[:, 0]
                                      + 2.0 ** -23 * loss_r, 0.0))
    assert lib.lb_train_status() == lib.LB_OK


def test_cross_entropy_gradient_against_differences(lib):
    """Along random directions, against central differences of the 64-bit objective (error about step^2)."""
    M, D, V = 40, 64, 300
    H, W, labels = _loss_inputs(9, M, D, V)
    weight = torch.rand(M, generator=_gen(2), device="cuda") / M
    _, dH, dW = lib.lb_cross_entropy_gradient(H, W, labels, weight)
    G, eG, _ = _grad_bounds(H, W, labels, weight, D)

    def objective(Hd, Wd):
        z = Hd @ Wd.T
        ok = (labels >= 0) & (labels < V)
        at = torch.where(ok, labels, 0)[:, None]
        loss = torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]
        return (torch.where(ok, loss, 0.0) * weight.double()).sum()

    Hd, Wd, eps = H.double(), W.double(), 1e-4
    for seed in range(4):
        g = _gen(100 + seed)
        U = torch.randn(M, D, generator=g, device="cuda", dtype=torch.float64)
        X = torch.randn(V, D, generator=g, device="cuda", dtype=torch.float64)
        dh = (objective(Hd + eps * U, Wd) - objective(Hd - eps * U, Wd)) / (2 * eps)
        dw = (objective(Hd, Wd + eps * X) - objective(Hd, Wd - eps * X)) / (2 * eps)
        bh = ((eG @ Wd.abs() * 1.01 + 2.0 ** -8 * (G @ Wd).abs() + 2.0 ** -18 * (G.abs() @ Wd.abs())) * U.abs()).sum()
        bw = ((eG.T @ Hd.abs() * 1.01 + 2.0 ** -8 * (G.T @ Hd).abs() + 2.0 ** -18 * (G.T.abs() @ Hd.abs())) * X.abs()).sum()
        assert abs(float((dH.double() * U).sum() - dh)) <= float(bh) + 1e-6
        assert abs(float((dW.double() * X).sum() - dw)) <= float(bw) + 1e-6


@pytest.mark.parametrize("M", [6, 200])
def test_cross_entropy_rows_that_do_not_count_and_nan_rows(lib, M):
    """NaN and infinity in a row that does not count reach nothing; in one that does, its own loss and row, and dW."""
    D, V = 64, 500
    H, W, labels = _loss_inputs(M, M, D, V)
    labels = labels.clamp(0, V - 1)
    labels[::3] = -100
    weight = torch.full((M,), 1.0 / M, device="cuda")
    clean = lib.lb_cross_entropy_gradient(H, W, labels, weight)
    H2 = H.clone()
    H2[0, 3] = float("nan")
    H2[3, :] = float("inf")
    loss, dH, dW = lib.lb_cross_entropy_gradient(H2, W, labels, weight)
    assert torch.equal(dW, clean[2]) and torch.equal(loss, clean[0]) and torch.equal(dH, clean[1])
    assert not dH[::3].any() and not loss[::3].any()
    l2, _ = lib.lb_cross_entropy_forward(H2, W, labels)
    assert torch.isfinite(l2).all() and not l2[::3].any()
    H2[1, 0] = float("nan")
    loss, dH, dW = lib.lb_cross_entropy_gradient(H2, W, labels, weight)
    others = torch.arange(M, device="cuda") != 1
    assert torch.isnan(loss[1]) and torch.isnan(dH[1]).all()
    assert torch.equal(loss[others], clean[0][others]) and torch.equal(dH[others], clean[1][others])
    l2, s2 = lib.lb_cross_entropy_forward(H2, W, labels)
    assert torch.isnan(l2[1]) and torch.isnan(s2[1]) and torch.isfinite(l2[others]).all()


def test_cross_entropy_nothing_counts(lib):
    M, D, V = 70, 64, 300
    H, W, _ = _loss_inputs(1, M, D, V)
    labels = torch.full((M,), -100, device="cuda")
    weight = torch.ones(M, device="cuda")
    loss, dH, dW = lib.lb_cross_entropy_gradient(H, W, labels, weight)
    assert not loss.any() and not dH.any() and not dW.any()
    labels[5] = 2                                                  # counts, with weight 0
    loss, dH, dW = lib.lb_cross_entropy_gradient(H, W, labels, torch.zeros_like(weight))
    assert float(loss[5]) > 0 and not dH.any() and not dW.any()
    e = lambda *s: torch.empty(*s, device="cuda")                  # noqa: E731
    loss, dH, dW = lib.lb_cross_entropy_gradient(H[:0], W, labels[:0], weight[:0])
    assert loss.shape == (0,) and dH.shape == (0, D) and not dW.any()
    loss, lse = lib.lb_cross_entropy_forward(H[:0], W, labels[:0])
    assert loss.shape == lse.shape == e(0).shape


def test_cross_entropy_sure_rows(lib):
    """A row that is sure of its label: p - 1 far below the rounding of p, so G must come from the logits."""
    M, D, V = 32, 128, 400
    g = _gen(5)
    W = (torch.randn(V, D, generator=g, device="cuda") * 0.2).to(BF16)
    labels = torch.arange(M, device="cuda") * 7
    w = W[labels].float()
    H = (9.0 * w / (w * w).sum(1, keepdim=True).sqrt()).to(BF16)
    weight = torch.full((M,), 1.0 / M, device="cuda")
    _, dH, dW = lib.lb_cross_entropy_gradient(H, W, labels, weight)
    G, eG, _ = _grad_bounds(H, W, labels, weight, D)
    p = 1.0 + G[torch.arange(M, device="cuda"), labels] * M
    assert float((1.0 - p).min()) < 1e-5
    # the label's entry: the error of p - 1 is that of the logits times p, not a rounding of p
    z, lse, _, _, at, mag = _loss_ref(H, W, labels)
    el = (_logit_bound(D, mag).gather(1, at)[:, 0] + _lse_bound(D, mag, z, lse)) / M
    eG.scatter_(1, at, (el + G.gather(1, at)[:, 0].abs() * 2.0 ** -8)[:, None])
    ref = G @ W.double()
    bound = eG @ W.double().abs() + 2.0 ** -17 * (G.abs() @ W.double().abs())
    _within(dH, ref, bound + 2.0 ** -8 * (ref.abs() + bound))


# ---------------------------------------------------------------------------------------------- orthogonalised updates

A, B, C = 3.4445, -4.7750, 2.0315


def _orth_ref(G, steps=5, eps=1e-7):
    X = G.double()
    wide = X.shape[0] < X.shape[1]
    X = X.T if wide else X
    X = X / (X.norm() + eps)
    for _ in range(steps):
        S = X.T @ X
        X = A * X + X @ (B * S + C * (S @ S))
    return X.T if wide else X


def _off(out, ref):
    return float((out.double() - ref).norm() / ref.norm())


# The rounding of the result is at most 2^-8 of it.  A_0 and the products after it are right to about 100 additions of
# 2^-22; a Gaussian matrix at least twice as long as wide has eigenvalues of A_0 within a factor of 34 of each other, and a
# direction moves by half the relative error of its eigenvalue: 34 / 2 * 100 * 2^-22 < 2^-11.
SMOOTH = 2.0 ** -8 + 2.0 ** -11


@pytest.mark.parametrize("shapes", [
    [(1, 1), (1, 5), (7, 1), (64, 16), (16, 64)],                 # one block each
    [(512, 16)] * 4 + [(24576, 1)],
    [(3000, 9), (9, 3000), (8191, 64)],                            # rank up to 64, long
    [(130, 65), (65, 130), (1001, 333), (200, 1500), (520, 260)],  # beyond, odd, both ways
    [(4096, 544)],
    [(5000, 2048)],
])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalise(lib, shapes, dtype):
    g = _gen(len(shapes))
    G = [(torch.randn(s, generator=g, device="cuda") * 10.0 ** (3 - 2 * i)).to(dtype) for i, s in enumerate(shapes)]
    for steps in (5, 1):
        out = lib.lb_orthogonalise(G, steps=steps)
        for X, O in zip(G, out):
            assert O.dtype == BF16 and O.shape == X.shape
            assert _off(O, _orth_ref(X, steps)) <= SMOOTH, tuple(X.shape)
    again = lib.lb_orthogonalise(G, steps=1)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert lib.lb_train_status() == lib.LB_OK


@pytest.mark.parametrize("m,n", [(1024, 256), (300, 300), (2000, 64), (600, 40)])
@pytest.mark.parametrize("kind", ["1/j", "1/j2", "1e-4", "spike", "rank"])
def test_orthogonalise_hard_spectra(lib, m, n, kind):
    """Singular values that fall off by 1e4 and more, one that dominates, and a matrix without full rank.  The small
    eigenvalues of A_0 are blown up by up to 485^2, so its errors are too; the bound allows them as much again as the
    rounding of the result, while one binary16 rounding of A_0 would give ten times that."""
    g = _gen(m + n)
    U, _ = torch.linalg.qr(torch.randn(m, n, generator=g, device="cuda", dtype=torch.float64))
    V, _ = torch.linalg.qr(torch.randn(n, n, generator=g, device="cuda", dtype=torch.float64))
    j = torch.arange(1, n + 1, device="cuda", dtype=torch.float64)
    s = {"1/j": 1 / j, "1/j2": 1 / j ** 2, "1e-4": 10.0 ** (-4 * (j - 1) / (n - 1)),
         "spike": torch.where(j == 1, 1.0, 0.002), "rank": torch.where(j <= n // 2, 1.0, 0.0)}[kind]
    G = ((U * s) @ V.T).float()
    out, = lib.lb_orthogonalise([G])
    assert _off(out, _orth_ref(G)) <= 2 * 2.0 ** -8


def _orth_bound(X, steps):
    """Rounding to bfloat16, and what the errors of the n x n part do to this matrix, to first order.

    Its symmetric operands are held to 2^-22 of their norm, and a product's truncated additions lose up to 1.5 * 2^-24 each,
    12 on the high halves of 128 k: together below 2^-20 of the norm.  An error E of A_k counts as E / a^(2k) of A_0, whose
    small eigenvalues grow by a^2 a step: the norms are max(lambda) at the start, at most 1.45 after, and T's roundings
    count 1 / a more: e = 2^-20 (max(lambda) + 1.45 (1 + 1 / a) / (a^2 - 1) + 0.1).  In the singular vectors' basis the
    result X_0 Q(A_0 + E) then moves by sigma_i E_ij (Q_i - Q_j) / (lambda_i - lambda_j), and no entry by more than twice
    the largest singular value of a result, 1.2."""
    a, b, c = 3.4445, -4.7750, 2.0315
    s0 = torch.linalg.svdvals(X.double())
    s0 = s0 / (s0.square().sum().sqrt() + 1e-7)
    lam0 = s0.square()
    lam, q, dlam, dq = lam0, torch.ones_like(s0), torch.ones_like(s0), torch.zeros_like(s0)
    for _ in range(steps):   # q = Q(lambda_0) and lambda = lambda_k with their derivatives by lambda_0
        f, df = a + b * lam + c * lam ** 2, (b + 2 * c * lam) * dlam
        q, dq = q * f, dq * f + q * df
        lam, dlam = lam * f ** 2, dlam * f ** 2 + 2 * lam * f * df
    gap = lam0[:, None] - lam0[None, :]
    near = gap.abs() <= 1e-6 * lam0[0]
    D = torch.where(near, dq[:, None], (q[:, None] - q[None, :]) / torch.where(near, 1.0, gap))
    e = 2.0 ** -20 * (lam0[0] + 1.45 * (1 + 1 / a) / (a * a - 1) + 0.1)
    moved = (s0[:, None] * D * e).abs().clamp(max=2.4)
    return 2.0 ** -8 + float(moved.norm() / (s0 * q).norm())


@pytest.mark.parametrize("steps", [1, 2, 3, 5, 10])
def test_orthogonalise_ranks_of_one_block(lib, steps):
    """Ranks 65 to 128, whose polynomial one block does: every edge inside its 32 x 32 blocks, few and many ranges of the
    long axis, and a batch.  Alone or together a matrix gives the same."""
    g = _gen(steps)
    shapes = [(n, n) for n in (65, 95, 97, 128)] + [(260, 127), (90, 1111), (20000, 66)] + [(700, 100)] * 5 + [(500, 129)]
    G = [torch.randn(s, generator=g, device="cuda") for s in shapes]
    out = lib.lb_orthogonalise(G, steps=steps)
    for i, (X, O) in enumerate(zip(G, out)):
        assert _off(O, _orth_ref(X, steps)) <= _orth_bound(X, steps), (i, tuple(X.shape))
    for i in (8, 3):
        assert torch.equal(out[i], lib.lb_orthogonalise([G[i]], steps=steps)[0])
    assert lib.lb_train_status() == lib.LB_OK


@pytest.mark.parametrize("kind", ["1/j", "1/j2", "1e-4", "spike", "rank"])
def test_orthogonalise_hard_spectra_of_one_block(lib, kind):
    test_orthogonalise_hard_spectra(lib, 1024, 120, kind)


@pytest.mark.parametrize("m,n", [(1 << 24, 2), (1 << 22, 130)])
def test_orthogonalise_longest(lib, m, n):
    """The longest sums of squares: a truncating accumulator must not shrink them.  At most 3 * 1024 additions of 1.5 * 2^-24
    scale A_0 by 1 - d, d <= 2.8e-4, and sigma by 1 - d / 2; the result's size then moves by sigma f'(sigma) d / 2 (the
    rounding to bfloat16 averages out over these many elements)."""
    a, b, c = 3.4445, -4.7750, 2.0315
    G = torch.randn(m, n, generator=_gen(m), device="cuda")
    out, = lib.lb_orthogonalise([G])
    X = G.double() / G.double().norm()
    A = X.T @ X
    lam = torch.linalg.eigvalsh(A)
    q, dq, l, dl = torch.ones_like(lam), torch.zeros_like(lam), lam, torch.ones_like(lam)
    one, Q = torch.eye(n, dtype=torch.float64, device="cuda"), torch.eye(n, dtype=torch.float64, device="cuda")
    for _ in range(5):
        p = a * one + b * A + c * A @ A
        Q, A = Q @ p, A @ p @ p
        f, df = a + b * l + c * l * l, (b + 2 * c * l) * dl
        q, dq = q * f, dq * f + q * df
        l, dl = l * f * f, dl * f * f + 2 * l * f * df
    ref = X @ Q
    bias = float(((out.double() - ref) * ref).sum() / ref.square().sum())
    moved = float((1 + 2 * lam * dq / q).abs().max()) * 2.8e-4 / 2
    assert abs(bias) <= moved + 2.0 ** -15, (bias, moved)


def test_orthogonalise_singular_values(lib):
    """What the update is for: five steps bring the singular values of a gradient-like matrix near 1."""
    g = _gen(8)
    G = torch.randn(900, 40, generator=g, device="cuda") @ torch.randn(40, 150, generator=g, device="cuda") \
        + 2.0 * torch.randn(900, 150, generator=g, device="cuda")
    out, = lib.lb_orthogonalise([G * 1e-6])
    s = torch.linalg.svdvals(out.double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


def test_orthogonalise_many_at_once(lib):
    """More matrices and more shapes than one set of launches takes, of every kind, each as if it were alone."""
    g = _gen(4)
    shapes = [(40 + 7 * i, 3 + i) for i in range(70)] + [(200 + 16 * i, 66 + 8 * i) for i in range(11)] + [(900, 70)] * 3 \
        + [(70, 700), (3000, 30), (2500, 30)]
    G = [torch.randn(s, generator=g, device="cuda") for s in shapes]
    out = lib.lb_orthogonalise(G)
    for i in (0, 33, 69, 70, 75, 80, 82, 84, 85, 86):
        assert torch.equal(out[i], lib.lb_orthogonalise([G[i]])[0]) or _off(out[i], _orth_ref(G[i])) <= SMOOTH
    for X, O in zip(G[70:], out[70:]):
        assert _off(O, _orth_ref(X)) <= 2 * 2.0 ** -8


@pytest.mark.parametrize("shape", [(96, 12), (5000, 20), (400, 100)])
def test_orthogonalise_zero_nan_scale(lib, shape):
    g = _gen(7)
    X = torch.randn(shape, generator=g, device="cuda")
    bad = X.clone()
    bad[3, 2] = float("nan")
    inf = X.clone()
    inf[0, 0] = float("inf")
    zero = torch.zeros_like(X)
    G = [X, bad, zero, inf, X * 1e-30, X * 1e30, X * 2.0 ** -140]
    out = lib.lb_orthogonalise(G, eps=0.0)
    ref = _orth_ref(X, eps=0.0)
    assert _off(out[0], ref) <= SMOOTH
    assert torch.isnan(out[1]).all() and torch.isnan(out[3]).all()
    assert not out[2].any()
    assert _off(out[4], ref) <= SMOOTH and _off(out[5], ref) <= SMOOTH    # the scale of a matrix does not matter
    # float32 itself has few bits left at 2^-140: against the matrix as it is stored
    assert _off(out[6], _orth_ref(G[6], eps=0.0)) <= SMOOTH
    small, = lib.lb_orthogonalise([X * 1e-12], eps=1e-7)                    # far below eps: linear, a^5 X / eps
    assert _off(small, _orth_ref(X * 1e-12)) <= SMOOTH


def test_orthogonalise_unaligned(lib):
    """Matrices one element past a 16-byte boundary; outputs of odd widths end at their last element."""
    g = _gen(6)
    for m, n in ((700, 70), (333, 77), (90, 10)):
        flat = torch.randn(m * n + 1, generator=g, device="cuda")
        G = flat[1:].view(m, n)
        buf = torch.full((m * n + 64,), -7.0, dtype=BF16, device="cuda")
        out = buf[1:1 + m * n].view(m, n)
        import ctypes
        vp, i = ctypes.c_void_p, ctypes.c_int
        ws = torch.empty(lib.lb_orthogonalise_workspace_bytes([(m, n)]) + 1, dtype=torch.uint8, device="cuda")
        st = lib._lib.lb_orthogonalise((vp * 1)(G.data_ptr()), lib.LB_F32, (i * 1)(m), (i * 1)(n), 1, 5, 1e-7,
                                       (vp * 1)(out.data_ptr()), ws.data_ptr(), ws.numel(),
                                       torch.cuda.current_stream().cuda_stream)
        assert st == lib.LB_OK
        assert _off(out, _orth_ref(G)) <= SMOOTH
        assert float(buf[0]) == -7.0 and bool((buf[1 + m * n:] == -7.0).all())


@pytest.mark.parametrize("rows,cols", [(65536, 72), (72, 65536), (16384, 800), (32768, 44)])
def test_orthogonalise_matrix_at_the_end_of_its_memory(lib, rows, cols):
    """Matrices that fill their 2 MB pages to the last byte, so that a read past the end is a read of unmapped memory."""
    assert rows * cols * 4 % (1 << 21) == 0 or cols == 44
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    G = torch.randn(rows, cols, generator=_gen(rows), device="cuda")
    out, = lib.lb_orthogonalise([G])
    assert _off(out, _orth_ref(G)) <= SMOOTH


# ---------------------------------------------------------------------------------------------- calls in earnest

def _all_calls(lib, seed):
    """One call of each operator; returns (call, inputs) with fixed outputs to compare."""
    g = _gen(seed)
    H, W, labels = _loss_inputs(seed, 200, 128, 1000)
    weight = torch.full((200,), 1 / 200, device="cuda")
    table = torch.randn(500, 96, generator=g, device="cuda")
    ids = _ids(g, (333,), 500)
    dout = torch.randn(333, 96, generator=g, device="cuda")
    mats = [torch.randn(300, 80, generator=g, device="cuda"), torch.randn(90, 20, generator=g, device="cuda"),
            torch.randn(4000, 24, generator=g, device="cuda")]

    def call(stream=None):
        return [lib.lb_embedding_forward(ids, table, stream=stream),
                lib.lb_embedding_backward(ids, dout, 500, stream=stream),
                *lib.lb_cross_entropy_forward(H, W, labels, stream=stream),
                *lib.lb_cross_entropy_forward(H[:9], W, labels[:9], stream=stream),
                *lib.lb_cross_entropy_gradient(H, W, labels, weight, stream=stream),
                *lib.lb_orthogonalise(mats, stream=stream)]
    return call, (H, W, labels, weight, table, ids, dout, *mats)


def test_captured_and_replayed(lib):
    call, inputs = _all_calls(lib, 1)
    want = [t.clone() for t in call()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # new values in the same buffers: a replay computes them anew
    call2, inputs2 = _all_calls(lib, 2)
    want2 = [t.clone() for t in call2()]
    for a, b in zip(inputs, inputs2):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want2, got))
    assert lib.lb_train_status() == lib.LB_OK


def test_two_streams_at_once(lib):
    """Calls on two streams that overlap on the device, each with its own scratch."""
    (c1, _), (c2, _) = _all_calls(lib, 1), _all_calls(lib, 2)
    want1, want2 = [t.clone() for t in c1()], [t.clone() for t in c2()]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    out1, out2 = [], []
    for _ in range(5):
        out1.append(c1(stream=s1))
        out2.append(c2(stream=s2.cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in out1 for a, b in zip(want1, out))
    assert all(torch.equal(a, b) for out in out2 for a, b in zip(want2, out))


def test_updates_of_every_kind_at_once(lib):
    """Matrices whose n x n part runs in one block (both ways), in a launch a product, or whole in one block, from two
    streams and a replayed graph that overlap, the same matrix twice in a list among them."""
    g = _gen(21)
    sets = [[torch.randn(s, generator=g, device="cuda") for s in shapes]
            for shapes in ([(700, 100), (90, 400), (300, 20), (900, 50), (600, 300)], [(256, 128)] * 3 + [(1500, 70), (400, 200)])]
    for G in sets:
        G.append(G[0])
    want = [[t.clone() for t in lib.lb_orthogonalise(G)] for G in sets]
    for W in want:
        assert torch.equal(W[0], W[-1])
    # results of equal shapes may share a storage, never an element, and each is contiguous
    apart = lib.lb_orthogonalise(sets[1] + [torch.ones(3, 5, device="cuda")] * 2)
    assert all(t.is_contiguous() for t in apart)
    ends = sorted((t.data_ptr(), t.data_ptr() + t.numel() * 2) for t in apart)
    assert all(a[1] <= b[0] for a, b in zip(ends, ends[1:]))
    graph, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        held = lib.lb_orthogonalise(sets[0])
    torch.cuda.synchronize()
    live, replayed = [], []
    for _ in range(4):
        with torch.cuda.stream(other):
            graph.replay()
            replayed.append([t.clone() for t in held])
        live.append((lib.lb_orthogonalise(sets[1], stream=side), lib.lb_orthogonalise(sets[0])))
    torch.cuda.synchronize()
    for out in replayed:
        assert all(torch.equal(a, b) for a, b in zip(want[0], out))
    for a, b in live:
        assert all(torch.equal(x, y) for x, y in zip(want[1] + want[0], a + b))
    assert lib.lb_train_status() == lib.LB_OK


def test_a_training_step(lib):
    """The operators as a step of a small model uses them: embedding, a LittleBit layer, the loss over the vocabulary with
    its gradients, back through the layer, the embedding's gradient, and orthogonalised updates of the latent factors;
    each gradient against the 64-bit formula's, evaluated at the values the step itself passed on."""
    V, K, N, r, M = 600, 96, 64, 24, 130
    g = _gen(11)
    table = torch.randn(V, K, generator=g, device="cuda").to(BF16)
    head = (torch.randn(V, N, generator=g, device="cuda") * 0.1).to(BF16)
    ids = torch.randint(0, V, (M,), generator=g, device="cuda")
    labels = torch.roll(ids, -1)
    labels[-1] = -100
    U = [torch.randn(N, r, generator=g, device="cuda") * 0.01 for _ in range(2)]
    Vl = [torch.randn(K, r, generator=g, device="cuda") * 0.01 for _ in range(2)]
    scale = lambda n: (torch.rand(n, generator=g, device="cuda") * 0.3 + 0.1).half()   # noqa: E731
    h, gg, l = ([scale(n) for _ in range(2)] for n in (N, K, r))
    packed = [lib.lb_pack_signs(u) for u in U], [lib.lb_pack_signs(v) for v in Vl]
    layer = lib.lb_layer_create(N, K, r, *packed, h, gg, l)
    back = lib.lb_backward_create(N, K, r, *packed, h, gg, l)

    x = lib.lb_embedding_forward(ids, table)
    y = lib.lb_linear_forward(x, layer)
    hidden = y.to(BF16)
    weight = (labels >= 0).float() / (labels >= 0).sum()
    loss, dhidden, dhead = lib.lb_cross_entropy_gradient(hidden, head, labels, weight)
    grads = lib.lb_layer_backward(back, x, dhidden.float(), U, Vl)
    dtable = lib.lb_embedding_backward(ids, grads["dx"], V)
    updates = lib.lb_orthogonalise(grads["dU"] + grads["dV"])

    G, eG, _ = _grad_bounds(hidden, head, labels, weight, N)
    ref = G @ head.double()
    bound = eG @ head.double().abs() + 2.0 ** -16 * (G.abs() @ head.double().abs())
    _within(dhidden, ref, bound + 2.0 ** -8 * (ref.abs() + bound))
    want = torch.zeros(V, K, dtype=torch.float64, device="cuda").index_add_(0, ids, grads["dx"].double())
    mag = torch.zeros(V, K, dtype=torch.float64, device="cuda").index_add_(0, ids, grads["dx"].double().abs())
    _within(dtable, want, M * 2.0 ** -24 * mag)
    for X, O in zip(grads["dU"] + grads["dV"], updates):
        assert _off(O, _orth_ref(X)) <= 2 * 2.0 ** -8
    assert lib.lb_train_status() == lib.LB_OK
    # a step along the updates lowers the loss to first order: <update, gradient> is the nuclear norm's order, positive
    for X, O in zip(grads["dU"] + grads["dV"], updates):
        assert float((X.double() * O.double()).sum()) > 0.5 * float(torch.linalg.svdvals(X.double()).sum())
