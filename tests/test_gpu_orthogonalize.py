"""Orthogonalised updates against the Newton-Schulz steps in 64 bits.

Bounds.  The result is rounded to bf16 once: at most 2^-8 of each entry, so of
the whole in the 2-norm.  Before that, matrices with min(N, K) <= 192 run on
22-bit operands and fp32 sums; what a step adds, some 2^-20 of X, the later
steps multiply by less than a^4 < 2^8 for directions not yet orthogonalised:
2^-12 in all.  Larger ones round R, Q and the products' X to fp16 (at most
2^-11 of each entry); how far that carries depends on the update, so the same
roundings are made in 64 bits (`_model`): the kernel and the model round
alike up to fp32 noise, and twice the model's distance from the exact result
is allowed on top.
"""
import pytest
import torch

import ternary_quantized_linear_b200 as tql

pytestmark = pytest.mark.gpu

DEFAULT = tql.ORTHOGONALIZE_COEFFICIENTS


def _update(B, N, K, kind, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    U = rand(B, N, K)
    if kind == "lowrank":
        U = 0.05 * U + rand(B, N, 4) @ rand(B, 4, K)
    elif kind == "rank1":
        U = rand(B, N, 1) * rand(B, 1, K)
    elif kind == "gaps":  # rows and columns of zeros
        U[:, ::3] = 0
        U[:, :, 1::4] = 0
    return (0.01 * U).to(dtype)


def _steps(X, rows, rnd):
    n = X.shape[-2]
    eye = torch.eye(n, dtype=X.dtype, device=X.device)
    for a, b, c in rows:
        H = rnd(X)
        A = H @ H.mT
        D = torch.diagonal(A, dim1=-2, dim2=-1)
        R = rnd(A * (1 - eye))
        R2 = R @ R
        Q = b * R + c * ((D[..., :, None] + D[..., None, :]) * R + R2)
        E = a + b * D + c * (D * D + torch.diagonal(R2, dim1=-2, dim2=-1))
        X = E[..., :, None] * X + rnd(Q * (1 - eye)) @ H
    return X


def _exact(U, rows, eps=1e-7, rnd=lambda t: t):
    X = U.double()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    if rnd is None:
        X = _steps(X, rows, lambda t: (t * 2.0 ** 12).half().double() * 2.0 ** -12)
    else:
        for a, b, c in rows:
            A = X @ X.mT
            X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT if tall else X


def _check(U, got, rows=None, eps=1e-7):
    rows = rows or [DEFAULT] * 5
    assert got.dtype == torch.bfloat16 and got.shape == U.shape
    e = _exact(U, rows, eps)
    size = torch.linalg.matrix_norm(e)
    tol = (2.0 ** -8 + 2.0 ** -12) * size
    if min(U.shape[-2:]) > 192:
        tol = tol + 2 * torch.linalg.matrix_norm(_exact(U, rows, eps, rnd=None) - e)
    off = torch.linalg.matrix_norm(got.double() - e)
    assert (off <= tol).all(), (off / size, tol / size)
    assert tql.bitnet_device_status(reset=False) == (tql.BITNET_OK, 0)


SHAPES = [(1, 1), (1, 7), (9, 1), (8, 8), (3, 300), (64, 64), (65, 63), (128, 128), (128, 129),
          (127, 257), (100, 640), (128, 2048), (2048, 128), (2047, 33), (128, 2049), (2056, 72),
          (129, 129), (192, 200), (193, 193), (200, 1001), (256, 256), (257, 300), (300, 257),
          (512, 1024), (1024, 513), (777, 2731), (1100, 1153), (1300, 1280), (2400, 2500)]


@pytest.mark.parametrize("kind", ["flat", "lowrank"])
@pytest.mark.parametrize("N,K", SHAPES)
def test_shapes(N, K, kind):
    U = _update(1, N, K, kind, torch.bfloat16 if (N + K) % 2 else torch.float32, seed=N + K)[0]
    _check(U, tql.bitnet_orthogonalize(U))


@pytest.mark.parametrize("kind", ["rank1", "gaps"])
@pytest.mark.parametrize("N,K", [(4, 4), (128, 500), (150, 150), (300, 700), (700, 300)])
def test_updates_without_full_rank(N, K, kind):
    U = _update(1, N, K, kind)[0]
    _check(U, tql.bitnet_orthogonalize(U))


@pytest.mark.parametrize("B,N,K", [(2, 5, 9), (7, 64, 100), (3, 100, 600), (20, 128, 2048),
                                   (5, 130, 70), (4, 200, 333), (3, 333, 200), (2, 600, 1000),
                                   (16, 256, 512)])
def test_stacks(B, N, K):
    U = _update(B, N, K, "lowrank", seed=B)
    U[1] *= 1e3  # each matrix has its own norm
    got = tql.bitnet_orthogonalize(U)
    _check(U, got)
    for b in (0, B - 1):  # and is computed by itself
        if min(N, K) <= 128:  # (larger ones may be cut into other tiles)
            assert torch.equal(tql.bitnet_orthogonalize(U[b].clone()), got[b])


@pytest.mark.parametrize("N,K", [(60, 90), (230, 400)])
def test_extreme_magnitudes(N, K):
    U = _update(1, N, K, "flat")[0]
    for s in (1e-30, 1e30):
        V = U * s
        _check(V, tql.bitnet_orthogonalize(V, eps=0.0), eps=0.0)
    # an update far below eps comes out small, as the formula has it
    V = U * 1e-9
    _check(V, tql.bitnet_orthogonalize(V, eps=1e-3), eps=1e-3)


@pytest.mark.parametrize("N,K", [(50, 70), (300, 260)])
def test_zero_and_non_finite(N, K):
    z = torch.zeros(N, K, device="cuda")
    assert (tql.bitnet_orthogonalize(z) == 0).all()
    assert (tql.bitnet_orthogonalize(z, eps=0.0) == 0).all()
    U = _update(3, N, K, "flat")
    want = tql.bitnet_orthogonalize(U)
    U[1, 3, 4] = float("nan")
    got = tql.bitnet_orthogonalize(U)
    assert torch.isnan(got[1]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    U[1, 3, 4] = float("inf")
    got = tql.bitnet_orthogonalize(U)
    assert torch.isnan(got[1]).all() and torch.equal(got[0], want[0])


def test_strided_and_misaligned_updates_are_refused():
    U = _update(1, 40, 64, "flat")[0]
    with pytest.raises(ValueError):
        tql.bitnet_orthogonalize(U.T)
    flat = torch.zeros(40 * 64 + 1, device="cuda")
    with pytest.raises(tql.BitnetError) as e:
        tql.bitnet_orthogonalize(flat[1:].view(40, 64))
    assert e.value.code == tql.BITNET_ERR_MISALIGNED
    empty = tql.bitnet_orthogonalize(torch.zeros(0, 40, 64, device="cuda"))
    assert empty.shape == (0, 40, 64)
    with pytest.raises(tql.BitnetError) as e:
        tql.bitnet_orthogonalize(torch.zeros(3, 0, device="cuda"))
    assert e.value.code == tql.BITNET_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("N,K", [(40, 100), (260, 300)])
@pytest.mark.parametrize("rows", [
    [DEFAULT],                                     # one step: the largest amplification alone
    [(1.5, -0.5, 0.0)] * 12,                       # cubic, converges to the polar factor
    [(15.0 / 8, -10.0 / 8, 3.0 / 8)] * 8,
    [(4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037)],
    [(2.0, 0.0, 0.0)] * 4,                         # grows: other scales each step
    [(0.25, 0.0, 0.0)] * 3,
])
def test_other_coefficients(N, K, rows):
    U = _update(1, N, K, "flat")[0]
    got = tql.bitnet_orthogonalize(U, steps=len(rows), coefficients=rows)
    _check(U, got, rows)


def test_polar_factor_is_orthogonal():
    # enough cubic steps: O O^T = 1 to the rounding of O, 2^-8 a row and its norm
    U = _update(1, 96, 200, "flat")[0]
    O = tql.bitnet_orthogonalize(U, steps=20, coefficients=(1.5, -0.5, 0.0)).double()
    eye = torch.eye(96, dtype=torch.float64, device="cuda")
    assert (O @ O.T - eye).abs().max() <= 2 * 2.0 ** -8 + 2.0 ** -12


def test_given_buffers_stay_inside():
    N, K = 300, 1001
    U = _update(1, N, K, "flat")[0]
    want = tql.bitnet_orthogonalize(U)
    nb = int(tql.load_library().bitnet_orthogonalize_workspace_bytes(1, N, K))
    ws = torch.full((nb + 512,), 7, dtype=torch.uint8, device="cuda")
    for k in (K, 1000):  # odd rows leave by plain stores, whole ones by TMA
        V = U[:, :k].contiguous()
        want = tql.bitnet_orthogonalize(V)
        flat = torch.full((N * k + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
        tql.bitnet_orthogonalize(V, out=flat[8:8 + N * k].view(N, k), workspace=ws[:nb])
        assert torch.equal(flat[8:8 + N * k].view(N, k), want)
        assert (flat[:8] == 3).all() and (flat[8 + N * k:] == 3).all()
    assert (ws[nb:] == 7).all()


@pytest.mark.parametrize("B,N,K", [(3, 100, 900), (1, 400, 700), (1, 1100, 600)])
def test_same_bits_on_streams_and_in_graphs(B, N, K):
    U, U2 = _update(B, N, K, "flat"), _update(B, N, K, "lowrank", seed=4)
    want, want2 = tql.bitnet_orthogonalize(U), tql.bitnet_orthogonalize(U2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a = tql.bitnet_orthogonalize(U, stream=s1)
        with torch.cuda.stream(s2):
            b = tql.bitnet_orthogonalize(U2)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want2)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    V = U.clone()
    with torch.cuda.graph(g1):
        a = tql.bitnet_orthogonalize(V)
    with torch.cuda.graph(g2):
        b = tql.bitnet_orthogonalize(U2)
    V.copy_(U2)
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        g1.replay()
    with torch.cuda.stream(s2):
        g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want2) and torch.equal(b, want2)


def test_a_training_step_together():
    """The warm-up layer, the head's loss, both backwards and the update of the
    layer's latent weights, as a training loop chains them."""
    M, V, N, K = 200, 1000, 256, 320
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    W, head = 0.05 * rand(N, K), (0.05 * rand(V, N)).bfloat16()
    x, t = rand(M, K), torch.randint(0, V, (M,), generator=g, device="cuda")
    t[::9] = -100
    count = (t >= 0).sum()
    dloss = (t >= 0).float() / count
    W_lam, _ = tql.bitnet_warmup_quantize_weights(W, 0.5)
    y, x_lam = tql.bitnet_warmup_forward(x, None, 1e-5, W_lam, 0.5, y_dtype=torch.bfloat16,
                                         keep_x_lam=True)
    loss, lse = tql.bitnet_cross_entropy_forward(y, head, t)
    dy, dhead = tql.bitnet_cross_entropy_backward(y, head, t, lse, dloss)
    _, dW = tql.bitnet_warmup_backward(dy, x_lam, W_lam, need_dx=False)
    O = tql.bitnet_orthogonalize(dW)
    # the same chain in 64 bits from each stage's own inputs
    z = y.double() @ head.double().T
    ok = t >= 0
    want = torch.nn.functional.cross_entropy(z[ok], t[ok])
    assert abs((loss.double() * dloss.double()).sum() - want) <= 1e-5 * want
    p = torch.softmax(z, 1)
    p[torch.arange(M, device="cuda"), t.clamp(min=0)] -= 1
    p *= dloss.double()[:, None]
    dy_want = p @ head.double()
    # g and dy rounded once each (2^-8 at most, in the 2-norm for entries of random sign)
    assert (dy.double() - dy_want).norm() <= 2 * 2.0 ** -8 * dy_want.norm()
    dW_want = dy.double().T @ x_lam.double()
    assert (dW.double() - dW_want).norm() <= 1e-5 * dW_want.norm()
    _check(dW, O)
    assert dhead.shape == head.shape


@pytest.mark.parametrize("B,N,K", [(1, 128, 4096), (1, 4096, 100), (2, 64, 3001), (1, 3, 2100),
                                   (14, 128, 2500), (15, 128, 2500), (1, 100, 4104),
                                   (1, 4100, 72), (1, 128, 8000)])
def test_long_and_narrow(B, N, K):
    """Clusters of sixteen (k up to 4096, more of them than fit at a time); past
    them products with both halves, cut along a long contraction."""
    U = _update(B, N, K, "lowrank", torch.bfloat16, seed=N + K)
    got = tql.bitnet_orthogonalize(U)
    for u, o in zip(U, got):
        _check(u, o)


@pytest.mark.parametrize("B,N,K", [(1, 100, 257), (7, 128, 1025), (8, 1025, 128), (15, 64, 512),
                                   (16, 64, 512), (34, 512, 40), (34, 20, 1024), (80, 33, 260)])
def test_every_cluster_of_small_updates(B, N, K):
    """Two to sixteen CTAs a matrix, by its columns and the batch."""
    U = _update(B, N, K, "flat", torch.float32, seed=B + N + K)
    got = tql.bitnet_orthogonalize(U)
    for u, o in zip(U, got):
        _check(u, o)


@pytest.mark.parametrize("N,K", [(40, 100), (160, 300), (260, 300)])
@pytest.mark.parametrize("rows", [
    [(0.1, 0.0, 0.0)] * 5,                          # bounds down to 2^-14 and 2^-17
    [(0.01, 0.0, 0.0)] * 3,
    [(1e-6, 0.0, 0.0), (0.5, -2.0 ** 38, 0.0)],     # a cubic that is felt at 2^-20
    [(0.001, 0.0, 0.0), (0.0, 1e6, 0.0)],           # and all of the next X
    [(1e-30, 0.0, 0.0)],                            # the last step may end anywhere
    [(1e-3, 0.0, 0.0)] * 8,                         # down to 2^-70, then 2^-80
    [(1e-6, 0.0, 0.0)] * 6 + [(1e6, 0.0, 0.0)] * 5,
    [(0.0, 0.0, 0.0)] * 2,
])
def test_shrinking_coefficients(N, K, rows):
    """Iterates that get small keep their digits: their scales follow them.
    (None of these steps multiplies what another one added by more than 3, so
    2^-12 covers 22 bits; above 192 rows the fp16 roundings again, here of
    entries relative to the largest.)"""
    U = _update(1, N, K, "flat")[0]
    got = tql.bitnet_orthogonalize(U, steps=len(rows), coefficients=rows)
    e = _exact(U, rows)
    size = torch.linalg.matrix_norm(e)
    tol = (2.0 ** -8 + 2.0 ** -12) * size
    if min(N, K) > 192:
        def half(t):
            unit = 2.0 ** -14 * t.abs().max().clamp(min=2.0 ** -300)
            return (t / unit).half().double() * unit
        X = U.double() / (torch.linalg.matrix_norm(U.double()) + 1e-7)
        tol = tol + 2 * torch.linalg.matrix_norm(_steps(X, rows, half) - e)
    assert torch.linalg.matrix_norm(got.double() - e) <= tol
    assert tql.bitnet_device_status(reset=False) == (tql.BITNET_OK, 0)


@pytest.mark.parametrize("B,N,K", [
    (1, 904, 1256), (1, 1256, 905),          # X X^T on clusters of three
    (1, 1179, 1621), (200, 1, 2054),         # of two
    (1, 195, 1106), (1, 3, 4100),            # of four
    (1, 130, 514),                           # of three, both halves
    (16, 389, 406), (40, 194, 200),          # SM pairs over a stack
    (40, 137, 137),                          # the same, both halves
    (8, 512, 1024),                          # single SMs, and pairs for the update
])
def test_every_cut_of_the_products(B, N, K):
    """A shape for each way that the products can be cut."""
    U = _update(B, N, K, "flat", torch.float32, seed=B + N + K)
    _check(U, tql.bitnet_orthogonalize(U))
