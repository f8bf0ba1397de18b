"""Host-side checks of the training operators (vocabulary cross entropy,
orthogonalised updates) that need no GPU: sizes, refusals through the C ABI
(fake pointers that are never dereferenced) and through the binding (CPU
tensors, which every check has to refuse before a pointer reaches the
library)."""
import ctypes

import pytest
import torch

import ternary_quantized_linear_b200 as tql
from ternary_quantized_linear_b200 import build as tql_build

FAKE = 0x10000
P = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    tql_build.build()
    return tql.load_library()


def _fwd(lib, x=FAKE, W=FAKE, t=FAKE, M=4, V=100, K=64, loss=FAKE, lse=FAKE, ws=FAKE, wsb=BIG):
    return lib.bitnet_cross_entropy_forward(P(x), P(W), P(t), M, V, K, P(loss), P(lse), P(ws), wsb,
                                            None)


def _bwd(lib, x=FAKE, W=FAKE, t=FAKE, lse=FAKE, dl=FAKE, M=4, V=100, K=64, dx=FAKE, dW=FAKE,
         ws=FAKE, wsb=BIG):
    return lib.bitnet_cross_entropy_backward(P(x), P(W), P(t), P(lse), P(dl), M, V, K, P(dx),
                                             P(dW), P(ws), wsb, None)


def _ortho(lib, U=FAKE, dt=0, B=1, N=300, K=400, steps=5, coef=None, eps=1e-7, O=FAKE, ws=FAKE,
           wsb=BIG, null_coef=False):
    coef = coef or [3.4445, -4.775, 2.0315] * max(steps, 1)
    arr = None if null_coef else (ctypes.c_double * len(coef))(*coef)
    return lib.bitnet_orthogonalize(P(U), dt, B, N, K, steps, arr, ctypes.c_float(eps), P(O),
                                    P(ws), wsb, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_cross_entropy_refuses_bad_arguments(lib, call):
    for bad in (dict(K=4), dict(K=12), dict(K=0), dict(V=0), dict(V=tql.BITNET_MAX_N + 1),
                dict(K=tql.BITNET_MAX_K + 8), dict(M=tql.BITNET_MAX_M + 1),
                dict(M=tql.BITNET_MAX_M, V=tql.BITNET_MAX_N)):
        assert call(lib, **bad) == tql.BITNET_ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(M=-1), dict(V=-1), dict(K=-8), dict(x=0), dict(W=0), dict(t=0), dict(lse=0)):
        assert call(lib, **bad) == tql.BITNET_ERR_INVALID_ARG, bad
    for bad in (dict(x=FAKE + 8), dict(W=FAKE + 8), dict(t=FAKE + 4), dict(lse=FAKE + 2),
                dict(ws=FAKE + 128)):
        assert call(lib, **bad) == tql.BITNET_ERR_MISALIGNED, bad
    assert call(lib, ws=0) == tql.BITNET_ERR_WORKSPACE
    assert call(lib, wsb=16) == tql.BITNET_ERR_WORKSPACE


def test_cross_entropy_outputs(lib):
    assert _fwd(lib, loss=0) == tql.BITNET_ERR_INVALID_ARG
    assert _bwd(lib, dl=0) == tql.BITNET_ERR_INVALID_ARG
    assert _fwd(lib, loss=FAKE + 1) == tql.BITNET_ERR_MISALIGNED
    assert _bwd(lib, dx=FAKE + 8) == tql.BITNET_ERR_MISALIGNED
    assert _bwd(lib, dW=FAKE + 8) == tql.BITNET_ERR_MISALIGNED
    # nothing asked for, or no tokens: queues nothing
    assert _bwd(lib, dx=0, dW=0) == tql.BITNET_OK
    assert _fwd(lib, M=0) == tql.BITNET_OK
    assert _bwd(lib, M=0, dW=0) == tql.BITNET_OK


def test_cross_entropy_workspaces(lib):
    f = lib.bitnet_cross_entropy_forward_workspace_bytes
    b = lib.bitnet_cross_entropy_backward_workspace_bytes
    for q in (f, b):
        assert q(0, 100, 64) == 0 and q(4, 100, 12) == 0 and q(-1, 100, 64) == 0
        assert q(5, 100, 64) % 256 == 0 and q(5, 100, 64) > 0
    # no logits: the forward keeps 8 bytes per token for each half tile
    assert f(8192, 128000, 4096) <= 8192 * (2 * 128000 // 128) * 8
    # the backward holds one piece of g (at most 256 MiB) and dx in fp32
    assert b(8192, 128000, 4096) < (256 << 20) + 2 * 4 * 8192 * 4096 + (1 << 20)
    for M, V, K in ((1, 1, 8), (1, 32000, 4096), (129, 257, 72), (3000, 50000, 64)):
        assert _fwd(lib, M=M, V=V, K=K, wsb=f(M, V, K) - 1) == tql.BITNET_ERR_WORKSPACE
        assert _bwd(lib, M=M, V=V, K=K, wsb=b(M, V, K) - 1) == tql.BITNET_ERR_WORKSPACE


def test_orthogonalize_refuses_bad_arguments(lib):
    for bad in (dict(N=0), dict(K=0), dict(N=tql.BITNET_MAX_K + 1), dict(B=65536),
                dict(B=60000, N=65536, K=65536)):
        assert _ortho(lib, **bad) == tql.BITNET_ERR_UNSUPPORTED_SHAPE, bad
    nan, inf = float("nan"), float("inf")
    for bad in (dict(N=-1), dict(B=-1), dict(U=0), dict(O=0), dict(dt=2), dict(steps=0),
                dict(steps=33), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
                dict(null_coef=True), dict(coef=[nan, 0, 0] * 5), dict(coef=[1, inf, 0] * 5),
                # diverges: singular values would pass 2^20
                dict(coef=[100.0, 0.0, 0.0] * 5)):
        assert _ortho(lib, **bad) == tql.BITNET_ERR_INVALID_ARG, bad
    for bad in (dict(U=FAKE + 8), dict(O=FAKE + 8), dict(ws=FAKE + 128)):
        assert _ortho(lib, **bad) == tql.BITNET_ERR_MISALIGNED, bad
    assert _ortho(lib, ws=0) == tql.BITNET_ERR_WORKSPACE
    need = lib.bitnet_orthogonalize_workspace_bytes(1, 300, 400)
    assert need > 0 and need % 256 == 0
    assert _ortho(lib, wsb=need - 1) == tql.BITNET_ERR_WORKSPACE
    assert _ortho(lib, B=0) == tql.BITNET_OK
    # what runs in shared memory needs no workspace
    assert lib.bitnet_orthogonalize_workspace_bytes(7, 128, 2048) == 0
    assert lib.bitnet_orthogonalize_workspace_bytes(7, 2048, 128) == 0
    assert lib.bitnet_orthogonalize_workspace_bytes(1, 129, 129) > 0
    assert lib.bitnet_orthogonalize_workspace_bytes(14, 4096, 128) == 0
    assert lib.bitnet_orthogonalize_workspace_bytes(15, 4096, 128) > 0
    assert lib.bitnet_orthogonalize_workspace_bytes(1, 128, 4097) > 0
    assert lib.bitnet_orthogonalize_workspace_bytes(1, 0, 5) == 0


def test_binding_refuses_wrong_tensors(lib):
    M, V, K = 4, 100, 64
    x, W = torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(V, K, dtype=torch.bfloat16)
    t = torch.zeros(M, dtype=torch.int64)
    s = torch.zeros(M)
    fwd, bwd, ort = (tql.bitnet_cross_entropy_forward, tql.bitnet_cross_entropy_backward,
                     tql.bitnet_orthogonalize)
    U = torch.zeros(8, 16)
    cases = [
        (ValueError, lambda: fwd(x, W, t)),                       # not on a GPU
        (ValueError, lambda: bwd(x, W, t, s, s)),
        (ValueError, lambda: ort(U)),
        (TypeError, lambda: fwd(x.float(), W, t)),
        (TypeError, lambda: fwd(x, W.half(), t)),
        (TypeError, lambda: fwd(x, W, t.int())),
        (ValueError, lambda: fwd(x, W, t[:3])),
        (ValueError, lambda: fwd(x[:, :56], W, t)),
        (ValueError, lambda: fwd(x[:, :4], W[:, :4], t)),
        (ValueError, lambda: fwd(x[0], W, t)),
        (ValueError, lambda: fwd(x, W, t, loss=s[:2])),
        (TypeError, lambda: fwd(x, W, t, lse=s.double())),
        (ValueError, lambda: fwd(x, W, t, workspace=torch.zeros(16, dtype=torch.uint8))),
        (TypeError, lambda: bwd(x, W, t, s.double(), s)),
        (ValueError, lambda: bwd(x, W, t, s, s[:1])),
        (ValueError, lambda: bwd(x, W, t, s, s, dx=torch.zeros(M, K - 8, dtype=torch.bfloat16))),
        (TypeError, lambda: bwd(x, W, t, s, s, dW=torch.zeros(V, K))),
        (TypeError, lambda: ort(U.half())),
        (ValueError, lambda: ort(U[0])),
        (ValueError, lambda: ort(U, steps=0)),
        (ValueError, lambda: ort(U, steps=33)),
        (ValueError, lambda: ort(U, coefficients=(1.0, 2.0))),
        (ValueError, lambda: ort(U, coefficients=[(1.0, 2.0, 3.0)] * 4)),
        (ValueError, lambda: ort(U, coefficients=[(1.0, 2.0)] * 5)),
        (TypeError, lambda: ort(U, out=torch.zeros(8, 16))),
        (ValueError, lambda: ort(U, out=torch.zeros(8, 8, dtype=torch.bfloat16))),
    ]
    for i, (exc, call) in enumerate(cases):
        with pytest.raises(exc):
            call()
