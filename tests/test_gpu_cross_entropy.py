"""Vocabulary cross entropy and its gradient against the formulas in 64 bits.

Bounds, with half steps 2^-24 (fp32) and 2^-8 (bf16):
* a logit is a sum of K exact products on the tensor cores, off by at most
  dz = (K/16 + 64) 2^-23 sum |x w| (the accumulation bound of the warm-up's
  tests: one truncated addition per 16 terms);
* exp is ex2 of a fused product, off by 2^-22 and by the rounding of the shift
  (z log2 e, twice: 2^-22 |z| covers it); a row's sum takes fewer than 200
  additions in any chain: e = dz + 2^-22 (1 + |z|max) + 200 * 2^-24;
* lse moves by at most e and two roundings of its size;
* loss = log(1 + s), s off by e and the target's own logit (a plain fp32 sum,
  (K/32 + 16) 2^-24 sum |x w| at most): min(1, s) times that, and its rounding;
* g: relative 2^-8 from bf16 and e from its exponential (at the target, where
  expm1 takes z_t - lse: e + the loss's error, absolute); a gradient sums
  |g| (2^-8 + e) |operand|, its fp32 sums (terms/16 + 64) 2^-23, and one
  rounding to bf16.
"""
import pytest
import torch

import ternary_quantized_linear_b200 as tql

pytestmark = pytest.mark.gpu


def _inputs(M, V, K, seed=0, sigma=0.05, ignored=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    W = (sigma * torch.randn((V, K), generator=g, device="cuda")).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    if ignored and M > 2:
        t[1::7] = -100
        t[2::11] = V  # one past the end: no target either
    d = torch.rand((M,), generator=g, device="cuda") - 0.3
    return x, W, t, d


def _exact(x, W, t, d):
    xd, Wd = x.double(), W.double()
    M, V, K = x.shape[0], W.shape[0], x.shape[1]
    z = xd @ Wd.T
    lse = torch.logsumexp(z, 1)
    ok = (t >= 0) & (t < V)
    at = torch.where(ok, t, 0)
    r = torch.arange(M, device=x.device)
    zt = z[r, at]
    others = z.clone()
    others[r, at] = -torch.inf
    loss = torch.where(ok, torch.log1p(torch.exp(others - zt[:, None]).sum(1)), 0.0)
    g = torch.exp(z - lse[:, None])
    g[r, at] = torch.where(ok, torch.expm1(zt - lse), 0.0)
    g = g * torch.where(ok, d.double(), 0.0)[:, None]
    out = {"lse": lse, "loss": loss, "dx": g @ Wd, "dW": g.T @ xd}
    # the bounds above
    absdot = (xd.abs() @ Wd.abs().T)
    dz = ((K / 16 + 64) * 2.0 ** -23 * absdot).amax(1)
    e = dz + 2.0 ** -22 * (1 + z.abs().amax(1)) + 200 * 2.0 ** -24
    et = (K / 32 + 16) * 2.0 ** -24 * absdot[r, at]
    s = torch.expm1(loss)
    tol = {"lse": e + et + 2.0 ** -23 * lse.abs(),
           "loss": torch.where(ok, s.clamp(max=1.0) * (e + et) + 2.0 ** -22 * loss, 0.0)}
    dg = g.abs() * (2.0 ** -8 + e[:, None])
    dg[r, at] += torch.where(ok, d.double().abs(), 0.0) * (e + et + 2.0 ** -22 * lse.abs())
    ga = g.abs()
    tol["dx"] = (dg + ga * (V / 16 + 64) * 2.0 ** -23) @ Wd.abs() + 2.0 ** -8 * out["dx"].abs()
    tol["dW"] = (dg + ga * (M / 16 + 64) * 2.0 ** -23).T @ xd.abs() + 2.0 ** -8 * out["dW"].abs()
    return out, tol


def _check(got, exact, tol, tiny=2.0 ** -126):
    for k, v in got.items():
        bad = (v.double() - exact[k]).abs() > tol[k] + tiny
        assert not bad.any(), (k, int(bad.sum()), (v.double() - exact[k]).abs().max().item())


def _run(x, W, t, d):
    loss, lse = tql.bitnet_cross_entropy_forward(x, W, t)
    dx, dW = tql.bitnet_cross_entropy_backward(x, W, t, lse, d)
    return {"loss": loss, "lse": lse, "dx": dx, "dW": dW}


SHAPES = [(1, 1, 8), (1, 2, 8), (1, 100, 64), (1, 5003, 520), (3, 31, 72), (5, 257, 64),
          (16, 40000, 64), (17, 33, 8), (64, 1000, 264), (127, 300, 64), (128, 256, 128),
          (129, 255, 136), (130, 3000, 72), (300, 5003, 520), (513, 999, 1000), (1025, 2049, 64),
          (2000, 700, 256), (4500, 1500, 64)]


@pytest.mark.parametrize("M,V,K", SHAPES)
def test_loss_and_gradient(M, V, K):
    x, W, t, d = _inputs(M, V, K, seed=M + V + K)
    exact, tol = _exact(x, W, t, d)
    _check(_run(x, W, t, d), exact, tol)
    assert tql.bitnet_device_status(reset=False) == (tql.BITNET_OK, 0)


def test_vocabulary_in_pieces():
    # g of 3000 tokens over 50000 entries passes the bytes of one piece
    M, V, K = 3000, 50000, 72
    x, W, t, d = _inputs(M, V, K, seed=5)
    t[-1], t[-3] = V - 1, 0
    exact, tol = _exact(x, W, t, d)
    _check(_run(x, W, t, d), exact, tol)


def test_vocabulary_in_pieces_without_slices():
    # dx has tiles enough for every SM: its pieces meet in the fp32 sum itself
    M, V, K = 5000, 27000, 2048
    x, W, t, d = _inputs(M, V, K, seed=6, sigma=0.02)
    exact, tol = _exact(x, W, t, d)
    _check(_run(x, W, t, d), exact, tol)


def test_confident_tokens_keep_their_digits():
    # targets far above the rest: losses down to 1e-12, never negative
    M, V, K = 200, 1000, 256
    x, W, t, d = _inputs(M, V, K, seed=2, ignored=False)
    lean = torch.linspace(0, 3, M, device="cuda")[:, None]
    x = (lean * W[t].float() / 0.05).bfloat16()
    d = torch.full_like(d, 1.0 / M)
    exact, tol = _exact(x, W, t, d)
    got = _run(x, W, t, d)
    assert (got["loss"] >= 0).all() and exact["loss"].min() < 1e-9
    _check(got, exact, tol)


def test_all_tokens_without_target():
    x, W, t, d = _inputs(40, 300, 64)
    t[:] = -100
    d[3] = float("nan")  # of a token without loss: not looked at
    got = _run(x, W, t, d)
    assert (got["loss"] == 0).all() and (got["dx"] == 0).all() and (got["dW"] == 0).all()
    exact, tol = _exact(x, W, t, torch.zeros_like(d))
    _check({"lse": got["lse"]}, exact, tol)


def test_zero_upstream_gradient_and_one_factor():
    x, W, t, d = _inputs(50, 300, 64)
    loss, lse = tql.bitnet_cross_entropy_forward(x, W, t)
    dx, dW = tql.bitnet_cross_entropy_backward(x, W, t, lse, torch.zeros_like(d))
    assert (dx == 0).all() and (dW == 0).all()
    # a power of two scales the gradient exactly
    a = tql.bitnet_cross_entropy_backward(x, W, t, lse, d)
    b = tql.bitnet_cross_entropy_backward(x, W, t, lse, d * 2.0 ** -20)
    assert torch.equal(a[0].float() * 2.0 ** -20, b[0].float())
    assert torch.equal(a[1].float() * 2.0 ** -20, b[1].float())


def test_large_and_equal_logits():
    M, V, K = 9, 700, 64
    x = torch.full((M, K), 4.0, device="cuda").bfloat16()
    W = torch.full((V, K), 0.5, device="cuda").bfloat16()     # every logit 128: lse = 128 + ln V
    W[0] = -64.0                                               # and one of -16384
    t = torch.arange(M, device="cuda")
    d = torch.ones(M, device="cuda")
    exact, tol = _exact(x, W, t, d)
    _check(_run(x, W, t, d), exact, tol)


def test_non_finite_rows_stay_their_own():
    x, W, t, d = _inputs(20, 300, 64, ignored=False)
    exact, tol = _exact(x, W, t, d)
    x = x.clone()
    x[4] = float("nan")
    x[9, 3] = float("inf")
    loss, lse = tql.bitnet_cross_entropy_forward(x, W, t)
    for m in (4, 9):
        assert not torch.isfinite(loss[m]) and not torch.isfinite(lse[m])
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[[4, 9]] = False
    assert ((loss.double() - exact["loss"]).abs() <= tol["loss"] + 1e-30)[keep].all()
    t2 = t.clone()
    t2[4] = -100
    loss, lse = tql.bitnet_cross_entropy_forward(x, W, t2)
    assert loss[4] == 0 and torch.isnan(lse[4])
    dx, _ = tql.bitnet_cross_entropy_backward(x, W, t2, lse, d, need_dW=False)
    assert (dx[4] == 0).all() and torch.isfinite(dx[keep]).all()


def test_no_tokens():
    x, W, _, _ = _inputs(1, 100, 64)
    x0, t0 = x[:0], torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = tql.bitnet_cross_entropy_forward(x0, W, t0)
    assert loss.shape == lse.shape == (0,)
    dW = torch.full_like(W, 7.0)
    dx, dW = tql.bitnet_cross_entropy_backward(x0, W, t0, lse, lse, dW=dW)
    assert dx.shape == x0.shape and (dW == 0).all()


def test_either_gradient_alone_and_given_buffers():
    x, W, t, d = _inputs(300, 1003, 520)
    loss, lse = tql.bitnet_cross_entropy_forward(x, W, t)
    dx, dW = tql.bitnet_cross_entropy_backward(x, W, t, lse, d)
    a, none = tql.bitnet_cross_entropy_backward(x, W, t, lse, d, need_dW=False)
    assert none is None and torch.equal(a, dx)
    none, b = tql.bitnet_cross_entropy_backward(x, W, t, lse, d, need_dx=False)
    assert none is None and torch.equal(b, dW)
    # rows around the outputs and the workspace's tail are left as they were
    big = torch.full((302, 520), 3.0, device="cuda").bfloat16()
    bigW = torch.full((1005, 520), 3.0, device="cuda").bfloat16()
    lib = tql.load_library()
    nb = int(lib.bitnet_cross_entropy_backward_workspace_bytes(300, 1003, 520))
    ws = torch.full((nb + 512,), 7, dtype=torch.uint8, device="cuda")
    tql.bitnet_cross_entropy_backward(x, W, t, lse, d, dx=big[1:301], dW=bigW[1:1004],
                                      workspace=ws[:nb])
    assert torch.equal(big[1:301], dx) and torch.equal(bigW[1:1004], dW)
    for edge in (big[0], big[301], bigW[0], bigW[1004]):
        assert (edge == 3.0).all()
    assert (ws[nb:] == 7).all()


@pytest.mark.parametrize("M,V,K", [(1, 32000, 256), (700, 5003, 264)])
def test_same_bits_on_streams_and_in_graphs(M, V, K):
    x, W, t, d = _inputs(M, V, K, seed=1)
    x2, _, t2, d2 = _inputs(M, V, K, seed=9)
    want, want2 = _run(x, W, t, d), _run(x2, W, t2, d2)
    torch.cuda.synchronize()
    # two calls under way at once
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = _run(x, W, t, d)
        with torch.cuda.stream(s2):
            b = _run(x2, W, t2, d2)
        loss, lse = tql.bitnet_cross_entropy_forward(x, W, t, stream=s1)
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], want[k]) for k in want)
        assert all(torch.equal(b[k], want2[k]) for k in want)
        assert torch.equal(loss, want["loss"]) and torch.equal(lse, want["lse"])
    # two captured graphs, replayed on new inputs and side by side
    xs, ts, ds = x.clone(), t.clone(), d.clone()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        a = _run(xs, W, ts, ds)
    with torch.cuda.graph(g2):
        b = _run(x2, W, t2, d2)
    xs.copy_(x2)
    ts.copy_(t2)
    ds.copy_(d2)
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        g1.replay()
    with torch.cuda.stream(s2):
        g2.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], want2[k]) for k in want)
    assert all(torch.equal(b[k], want2[k]) for k in want)


def test_gradient_against_differences():
    # x on a grid of 1/16, moved by h = 1/8 either way without rounding; the
    # third derivative of the loss along one coordinate is at most that of a
    # log-sum-exp over weights of range r: r^3, so the central difference is
    # off by h^2 r^3 / 6, and by the two losses' own errors over 2 h
    M, V, K, h = 6, 200, 64, 0.125
    x, W, t, _ = _inputs(M, V, K, seed=3, sigma=0.3, ignored=False)
    x = ((x.float() * 16).round() / 16).clamp(-2, 2).bfloat16()
    d = torch.ones(M, device="cuda")
    _, lse = tql.bitnet_cross_entropy_forward(x, W, t)
    dx, _ = tql.bitnet_cross_entropy_backward(x, W, t, lse, d)
    exact, tol = _exact(x, W, t, d)
    r = (W.float().amax(0) - W.float().amin(0)).double()
    for k in range(0, K, 7):
        up, dn = x.clone(), x.clone()
        up[:, k] += h
        dn[:, k] -= h
        assert torch.equal((up - dn)[:, k].float(), torch.full((M,), 2 * h, device="cuda"))
        diff = (tql.bitnet_cross_entropy_forward(up, W, t)[0].double()
                - tql.bitnet_cross_entropy_forward(dn, W, t)[0].double()) / (2 * h)
        allow = h * h * r[k] ** 3 / 6 + 4 * tol["loss"].max() / (2 * h) + tol["dx"][:, k]
        assert ((diff - dx[:, k].double()).abs() <= allow).all()


def test_cross_entropy_refuses_strided_tensors():
    x, W, t, _ = _inputs(4, 100, 64)
    with pytest.raises(ValueError):
        tql.bitnet_cross_entropy_forward(x.T.contiguous().T, W, t)
    with pytest.raises(tql.BitnetError) as e:
        flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
        tql.bitnet_cross_entropy_forward(flat[1:].view(4, 64), W, t)
    assert e.value.code == tql.BITNET_ERR_MISALIGNED


@pytest.mark.parametrize("M", [1, 100])
def test_few_rows_sum_in_short_runs(M):
    """All terms positive, so that truncated sums err one way: the tensor cores
    sum 512 terms at a time.  A run's 32 truncations lose less than 2^-23 of
    the sum so far each, 16.5 * 2^-23 of the run together; the eight runs join
    with seven roundings.  (4096 terms in one go would lose up to 128 * 2^-23,
    about a third of it in the mean.)"""
    V, K = 2000, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (0.5 + torch.rand((M, K), generator=g, device="cuda")).bfloat16()
    W = (0.005 + 0.01 * torch.rand((V, K), generator=g, device="cuda")).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    lse = tql.bitnet_cross_entropy_forward(x, W, t)[1].double()
    z = x.double() @ W.double().T
    exact = torch.logsumexp(z, 1)
    # the target's own logit (K/32 + 16 roundings) counts by its share of the sum
    share = torch.exp(z.amax(1) - exact) * (K / 32 + 16) * 2.0 ** -24
    tol = (z.amax(1) * (16.5 * 2.0 ** -23 + 7 * 2.0 ** -24 + share) + 2.0 ** -23 * exact
           + 2.0 ** -22 * (1 + z.amax(1)) + 200 * 2.0 ** -24)
    assert ((lse - exact).abs() <= tol).all(), ((lse - exact).abs() / tol).max()


@pytest.mark.parametrize("M,V,K", [(1, 90000, 1032), (64, 40001, 1544), (128, 39000, 1024),
                                   (200, 700, 1096)])
def test_runs_over_several_tiles(M, V, K):
    """More tiles than SMs, each of more than one run (the last one short)."""
    x, W, t, d = _inputs(M, V, K, seed=M + V, sigma=0.02)
    exact, tol = _exact(x, W, t, d)
    _check(_run(x, W, t, d), exact, tol)
    assert tql.bitnet_device_status(reset=False) == (tql.BITNET_OK, 0)


def _close(got, exact, tol, tiny=2.0 ** -126):
    """As _check, and a NaN is never close."""
    for k, v in got.items():
        off = (v.double() - exact[k]).abs()
        assert (off <= tol[k] + tiny).all(), (k, off.max().item())


@pytest.mark.parametrize("M,V,K", [(40, 300, 64), (300, 5003, 520)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_upstream_gradients_stay_their_own(M, V, K, bad):
    x, W, t, d = _inputs(M, V, K, seed=M)  # (tokens 1, 8, ... have no target)
    exact, tol = _exact(x, W, t, d)
    loss, lse = tql.bitnet_cross_entropy_forward(x, W, t)
    d = d.clone()
    d[[5, 20]] = bad
    d[1] = bad  # of a token without loss: not looked at
    dx, _ = tql.bitnet_cross_entropy_backward(x, W, t, lse, d, need_dW=False)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[5, 20]] = False
    _close({"dx": dx[keep]}, {"dx": exact["dx"][keep]}, {"dx": tol["dx"][keep]})
    assert (dx[(t < 0) | (t >= V)] == 0).all()
    assert not torch.isfinite(dx[5]).any() and not torch.isfinite(dx[20]).any()
    # nothing finite but zeros: those rows still have no gradient
    dx, _ = tql.bitnet_cross_entropy_backward(x, W, t, lse, torch.where(keep, 0.0, bad),
                                              need_dW=False)
    assert (dx[keep] == 0).all() and not torch.isfinite(dx[~keep]).any()


@pytest.mark.parametrize("M,V,K", [(7, 300, 64), (300, 700, 72)])
def test_infinite_logits(M, V, K):
    """An entry whose logit is -inf for every token has no weight: as if the
    vocabulary ended before it; as the target its loss is inf, by the formula
    with lse as it is, and its gradient -1.  A target at +inf gives inf - inf."""
    x, W, t, d = _inputs(M, V, K, seed=V, ignored=False)
    x[:, 0] = x[:, 0].abs() + 0.5
    at = V - 1
    t[t == at] = 0
    exact, tol = _exact(x, W[:at], t, d)
    Wm = W.clone()
    Wm[at, 0] = -torch.inf
    loss, lse = tql.bitnet_cross_entropy_forward(x, Wm, t)
    _close({"loss": loss, "lse": lse}, exact, tol)
    _, dW = tql.bitnet_cross_entropy_backward(x, Wm, t, lse, d, need_dx=False)
    _close({"dW": dW[:at]}, exact, tol)
    assert (dW[at] == 0).all()
    t2 = t.clone()
    t2[2] = at
    loss, lse = tql.bitnet_cross_entropy_forward(x, Wm, t2)
    assert loss[2] == torch.inf
    _close({"lse": lse}, exact, tol)
    # g of that row is dloss (softmax - onehot), the onehot at an entry of no weight
    only = torch.zeros_like(d)
    only[2] = 1.0
    _, dW = tql.bitnet_cross_entropy_backward(x, Wm, t2, lse, only, need_dx=False)
    assert torch.equal(dW[at], -x[2])
    Wp = W.clone()
    Wp[at, 0] = torch.inf
    loss, lse = tql.bitnet_cross_entropy_forward(x, Wp, t2)
    assert not torch.isfinite(lse).any() and torch.isnan(loss[2])
    assert not torch.isfinite(loss).any()


@pytest.mark.parametrize("M,V,K", [(129, 40000, 4096), (300, 20000, 4096), (1000, 9000, 2184)])
def test_many_rows_sum_in_short_runs(M, V, K):
    """As test_few_rows_sum_in_short_runs, on SM pairs: terms of one sign, of
    which the tensor cores sum 1024 at a time: 64 truncations, 32.5 * 2^-23 of
    the run together, and a rounding where it joins the others.  The loss, log(1 + sum e^(z_v - z_t)),
    takes z_t from a sum of K/32 rounded terms in a lane and the join of the
    lanes: partial sums of one sign grow evenly, so half of the roundings count."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (0.5 + torch.rand((M, K), generator=g, device="cuda")).bfloat16()
    W = (0.005 + 0.01 * torch.rand((V, K), generator=g, device="cuda")).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    loss, lse = (v.double() for v in tql.bitnet_cross_entropy_forward(x, W, t))
    z = x.double() @ W.double().T
    top = z.amax(1)
    exact = torch.logsumexp(z, 1)
    runs = -(-K // 1024)
    e = (top * (32.5 * 2.0 ** -23 + (runs - 1) * 2.0 ** -24) + 2.0 ** -22 * (1 + top)
         + 200 * 2.0 ** -24)
    target = top * (0.55 * K / 32 + 5) * 2.0 ** -24
    share = torch.exp(top - exact)
    assert ((lse - exact).abs() <= e + share * target + 2.0 ** -23 * exact).all(), \
        ((lse - exact).abs() / e).max()
    want = exact - z[torch.arange(M, device="cuda"), t]
    assert ((loss - want).abs() <= e + target + 2.0 ** -22 * want).all(), \
        ((loss - want).abs() / e).max()


def _busy(stream):
    """Hold `stream` for some 50 ms."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


@pytest.mark.parametrize("op", ["forward", "backward", "orthogonalize"])
def test_temporaries_given_to_another_stream(op):
    """An input that the caller lets go of while the other stream has not come
    to it yet stays allocated until that stream has read it."""
    M, V, K = 1024, 2000, 1024
    x, W, t, d = _inputs(M, V, K, seed=8)
    want = _run(x, W, t, d)
    U = W.float()
    o_want = tql.bitnet_orthogonalize(U)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(s)
    if op == "forward":
        got = tql.bitnet_cross_entropy_forward(x.clone(), W.clone(), t.clone(), stream=s)
        pairs = [(got[0], want["loss"]), (got[1], want["lse"])]
    elif op == "backward":
        got = tql.bitnet_cross_entropy_backward(x.clone(), W.clone(), t.clone(),
                                                want["lse"].clone(), d.clone(), stream=s)
        pairs = [(got[0], want["dx"]), (got[1], want["dW"])]
    else:
        pairs = [(tql.bitnet_orthogonalize(U.clone(), stream=s), o_want)]
    # what the allocator hands out now on the current stream is written at once
    again = [torch.zeros_like(v) for v in (x, W, t, d, U) for _ in range(16)]
    torch.cuda.synchronize()
    assert len(again) == 80 and all(torch.equal(a, b) for a, b in pairs)


@pytest.mark.parametrize("M,V,K", [(300, 40001, 1544), (1500, 20003, 1032), (129, 45000, 2056)])
def test_runs_of_pairs_over_several_tiles(M, V, K):
    """More 256 x 256 tiles than SM pairs, each of more than one run of 1024
    terms (the last one short): loss and gradient."""
    x, W, t, d = _inputs(M, V, K, seed=M + V, sigma=0.02)
    exact, tol = _exact(x, W, t, d)
    _close(_run(x, W, t, d), exact, tol)
    assert tql.bitnet_device_status(reset=False) == (tql.BITNET_OK, 0)


@pytest.mark.parametrize("M,V,K", [(1, 90001, 64), (1, 5003, 1032), (100, 40001, 64),
                                   (128, 33000, 72), (200, 21000, 64), (300, 2049, 520)])
def test_every_edge_column_counts_once(M, V, K):
    """One entry far above the rest, at either side of every kind of edge (a
    chunk of 32 columns, a tile of any width, the last column): left out or
    counted twice it would move lse by ln 2 at least."""
    g = torch.Generator(device="cuda").manual_seed(M + V)
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, 0] = 1.0
    x = x.bfloat16()
    W = (0.01 * torch.randn((V, K), generator=g, device="cuda")).bfloat16()
    W[:, 0] = 0.0
    t = torch.full((M,), V // 2 + 1, device="cuda")
    cols = {0, 1, V - 1, V - 2}
    for width in range(16, 272, 16):       # tiles are a multiple of 16 columns wide
        for n in (1, 2, V // width // 2, V // width):
            cols |= {n * width - 1, n * width}
    cols |= {c for c in range(0, min(V, 1056))}
    for c in sorted(c for c in cols if 0 <= c < V and c != V // 2 + 1):
        old = W[c, 0].clone()
        W[c, 0] = 30.0                      # e^30 against e^(+-1) of all others
        _, lse = tql.bitnet_cross_entropy_forward(x, W, t)
        W[c, 0] = old
        z = 30.0 + (x[:, 1:].double() @ W[c, 1:].double())
        # the others' share is below V e^-28; z itself, 30 and some +-10 of small
        # terms, is within (K/16 + 64) 2^-23 * 40 < 7e-4
        assert ((lse.double() - z).abs() <= 1e-3).all(), (c, (lse.double() - z).abs().max())


def test_overlapping_buffers_are_refused():
    M, V, K = 40, 300, 64
    x, W, t, d = _inputs(M, V, K)
    loss, lse = tql.bitnet_cross_entropy_forward(x, W, t)
    both = torch.empty(M + 1, device="cuda")
    big = torch.empty(V + M, K, dtype=torch.bfloat16, device="cuda")
    square = torch.randn(256, 256, device="cuda").bfloat16()
    scratch = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    for call in (
            lambda: tql.bitnet_cross_entropy_forward(x, W, t, loss=both[:M], lse=both[1:]),
            lambda: tql.bitnet_cross_entropy_backward(x, W, t, lse, d, dx=x),
            lambda: tql.bitnet_cross_entropy_backward(x, W, t, lse, d, dW=W),
            lambda: tql.bitnet_cross_entropy_backward(x, W, t, lse, d, dx=big[V - 1:V + M - 1],
                                                      dW=big[:V]),
            lambda: tql.bitnet_orthogonalize(square, out=square),
            lambda: tql.bitnet_orthogonalize(scratch[:1 << 16].view(torch.float32).view(128, 128),
                                             workspace=scratch)):
        with pytest.raises(ValueError):
            call()
    # neighbours do not overlap
    dx, dW = tql.bitnet_cross_entropy_backward(x, W, t, lse, d, dx=big[V:], dW=big[:V])
    want = _run(x, W, t, d)
    assert torch.equal(dx, want["dx"]) and torch.equal(dW, want["dW"])


def test_same_bits_in_runs_on_pairs():
    test_same_bits_on_streams_and_in_graphs(300, 20000, 1032)


@pytest.mark.parametrize("M,V,K", SHAPES)
def test_results_are_finite(M, V, K):
    assert all(torch.isfinite(v).all() for v in _run(*_inputs(M, V, K, seed=M + V + K)).values())
