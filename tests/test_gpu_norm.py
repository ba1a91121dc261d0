"""aa_layernorm_fwd and aa_layernorm_bwd against the definitions in float64.
Needs an MI355X.

Tolerances.  u = 2^-24 is half a step of float32 relative to the value.  A row
sum runs over at most 32 terms of a lane, then 6 butterfly steps and up to 16
waves, so its error is at most 64 u times the sum of the magnitudes; the few
single operations behind it are counted into the same 64.  With a = mean |x|:
  mean       |err| <= 64 u a
  rstd       relative 64 u, plus what the mean's error does to the variance:
             (64 u a)^2 rstd^2 / 2, which is below u for the data here
  y          |gamma| rstd (64 u a + 64 u |x - mean|) + 4 u (|y| + |beta|)
  dx         rstd (64 u (|g| + mean |g| + |xh| mean |g xh|)) and, as xh is off by
             64 u (|xh| + a rstd), |xh| enters with that error too
  dgamma     the sum over M rows: in one workgroup and the join at most M terms
             in a row, M u sum |dy xh|, and xh's own error
and every output adds half a step of its type: 2^-9 |value| for bf16 twice
over (eps / 2 = 2^-8 relative to the value), 2^-24 for float32.
"""
import numpy as np
import pytest
import torch

import associative_algebra_block_amd as aa
from tests._gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def half_step(t):
    return torch.finfo(t).eps / 2


def make(M, d, dtype, seed, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, d, generator=g) * (0.2 + torch.rand(d, generator=g)) + offset
    return x.to(dtype).to(DEV), g


def rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def guarded(shape, dtype):
    """A dense view inside a buffer of a known value, and the buffer."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), 77.0, dtype=dtype, device=DEV)
    return buf[64:64 + n].view(shape), buf


def untouched(buf):
    return bool((buf[:64] == 77.0).all()) and bool((buf[-64:] == 77.0).all())


def close(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    worst = float((err / tol.clamp_min(1e-300)).max()) if err.numel() else 0.0
    say(f"{what}: worst error / bound {worst:.3f}")
    assert bool((err <= tol).all()), (what, worst)


def reference(x, gamma, beta, eps):
    x = x.double().cpu()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    g = torch.ones(x.shape[1], dtype=torch.float64) if gamma is None else gamma.double().cpu()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if beta is None else beta.double().cpu()
    return x, mean, rstd, xh, g, b


# widths at each split's edges (256, 512, 768, 1024, 2048, 4096, 8192, 16384), odd ones among them
SIZES = [(1, 1), (3, 2), (1, 3), (5, 7), (2, 64), (9, 255), (4, 256), (7, 257), (3, 511), (6, 513), (1, 768), (37, 768),
         (5, 769), (11, 1024), (10, 1025), (3, 2047), (8, 2048), (5, 2049), (2, 4096), (3, 4097), (2, 8192), (3, 8193),
         (1, 16383), (2, 16384), (4200, 768), (2111, 100), (600, 4100),
         (9000, 1030)]   # outputs of more than 32 MB, which go past the caches


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("xt,yt,delta", [(F32, BF16, None), (F32, F32, BF16), (BF16, BF16, BF16), (BF16, F32, F32),
                                         (F32, BF16, F32)])
def test_forward(M, d, xt, yt, delta):
    say("norm fwd", M, d, xt, yt, delta)
    X, g = make(M, d, xt, 17 * d + M)
    gamma, beta = rand(g, (d,), F32), rand(g, (d,), F32)
    D = None if delta is None else rand(g, (M, d), delta)
    Y, ybuf = guarded((M, d), yt)
    S, sbuf = guarded((M, d), xt) if D is not None else (None, None)
    mean, mbuf = guarded((M,), F32)
    rstd, rbuf = guarded((M,), F32)
    eps = 1e-5
    aa.aa_layernorm_fwd(X, gamma, beta, Y, D, S, mean, rstd, eps)
    torch.cuda.synchronize()
    src = X
    if D is not None:
        want = (X.float() + D.float()).to(xt)
        assert torch.equal(S, want)
        src = S
    x, m, r, xh, gm, b = reference(src, gamma, beta, eps)
    a = x.abs().mean(1, keepdim=True)
    close(mean, m[:, 0], (64 * U * a + 1e-30)[:, 0], "mean")
    close(rstd, r[:, 0], (65 * U * r + 0.5 * (64 * U * a) ** 2 * r ** 3)[:, 0], "rstd")
    y = xh * gm + b
    tol = gm.abs() * r * 64 * U * (a + (x - m).abs()) + 65 * U * (gm * xh).abs() + 4 * U * (y.abs() + b.abs())
    close(Y, y, tol + half_step(yt) * (y.abs() + tol), "y")
    assert untouched(ybuf) and untouched(mbuf) and untouched(rbuf)
    assert sbuf is None or untouched(sbuf)


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("xt,dyt,ds", [(F32, BF16, True), (BF16, BF16, False), (BF16, F32, True), (F32, F32, False)])
def test_backward(M, d, xt, dyt, ds):
    say("norm bwd", M, d, xt, dyt, ds)
    X, g = make(M, d, xt, 31 * d + M)
    gamma = rand(g, (d,), F32)
    dY = rand(g, (M, d), dyt)
    dS = rand(g, (M, d), xt) if ds else None
    eps = 1e-5
    x, m, r, xh, gm, _ = reference(X, gamma, None, eps)
    mean, rstd = m[:, 0].float().to(DEV), r[:, 0].float().to(DEV)
    dX, xbuf = guarded((M, d), xt)
    dG, gbuf = guarded((d,), F32)
    dB, bbuf = guarded((d,), F32)
    nb = aa.aa_layernorm_bwd_workspace(M, d)
    ws = torch.full((nb + 256,), 85, dtype=torch.uint8, device=DEV)
    aa.aa_layernorm_bwd(X, dY, gamma, mean, rstd, dX, dG, dB, dS, ws[:nb])
    torch.cuda.synchronize()
    assert bool((ws[nb:] == 85).all())
    dy = dY.double().cpu()
    gg = dy * gm
    c1, c2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    dx = r * (gg - c1 - xh * c2)
    if ds:
        dx = dx + dS.double().cpu()
    a = x.abs().mean(1, keepdim=True)
    exh = 64 * U * (xh.abs() + a * r)                       # error of xh (its mean and rstd are rounded)
    tol = r * (64 * U * (gg.abs() + gg.abs().mean(1, keepdim=True) + xh.abs() * (gg * xh).abs().mean(1, keepdim=True))
               + exh * c2.abs() + xh.abs() * (gg.abs() * exh).mean(1, keepdim=True)) + 4 * U * dx.abs()
    close(dX, dx, tol + half_step(xt) * (dx.abs() + tol), "dx")
    n = (M + 64) * U
    close(dG, (dy * xh).sum(0), n * (dy * xh).abs().sum(0) + (dy.abs() * exh).sum(0) + 1e-30, "dgamma")
    close(dB, dy.sum(0), n * dy.abs().sum(0) + 1e-30, "dbeta")
    assert untouched(xbuf) and untouched(gbuf) and untouched(bbuf)


@pytest.mark.parametrize("M,d", [(1, 768), (3, 5), (5, 1025), (257, 2049), (1003, 2047), (2300, 8192), (600, 16383),
                                 (4600, 2048), (9000, 1030), (12288, 768), (12289, 1024), (20001, 300), (65537, 64)])
@pytest.mark.parametrize("xt,dyt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_every_row_counts_once_in_the_weights_gradients(M, d, xt, dyt):
    """Small whole numbers with mean 0 and rstd 1: xh is X, every product and sum
    is a whole number below 2^24 (9 M at most), so the sums are exact in any
    order and a row lost or taken twice shows in every column that it touches."""
    assert 9 * M < 1 << 24
    say("norm bwd exact", M, d, xt, dyt)
    g = torch.Generator().manual_seed(M + d)
    X, dY = (torch.randint(-3, 4, (M, d), generator=g) for _ in range(2))
    dY += (dY == 0) * 2                                      # no row is silent
    mean, rstd = torch.zeros(M, device=DEV), torch.ones(M, device=DEV)
    dX = torch.empty(M, d, dtype=xt, device=DEV)
    dG, dB = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.full((aa.aa_layernorm_bwd_workspace(M, d),), 255, dtype=torch.uint8, device=DEV)
    aa.aa_layernorm_bwd(X.to(xt).to(DEV), dY.to(dyt).to(DEV), None, mean, rstd, dX, dG, dB, None, ws)
    assert torch.equal(dG.cpu().long(), (X * dY).sum(0)) and torch.equal(dB.cpu().long(), dY.sum(0))


def test_gradient_formula_against_differences():
    """The formula that the tests above hold the kernel to, against central
    differences of the forward definition in float64 (step 1e-5: truncation
    about 1e-10, rounding about 1e-11 relative to the loss)."""
    g = torch.Generator().manual_seed(5)
    M, d, eps = 3, 9, 1e-5
    x, w = torch.randn(M, d, generator=g).double(), torch.randn(M, d, generator=g).double()
    gamma, beta = torch.randn(d, generator=g).double(), torch.randn(d, generator=g).double()

    def loss(x, gamma, beta):
        mu = x.mean(1, keepdim=True)
        xh = (x - mu) / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + eps)
        return float(((xh * gamma + beta) * w).sum())

    X = x.float().to(DEV)
    x = X.double().cpu()
    _, m, r, _, _, _ = reference(X, None, None, eps)
    dX, dG, dB = torch.empty_like(X), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(aa.aa_layernorm_bwd_workspace(M, d), dtype=torch.uint8, device=DEV)
    aa.aa_layernorm_bwd(X, w.float().to(DEV), gamma.float().to(DEV), m[:, 0].float().to(DEV),
                        r[:, 0].float().to(DEV), dX, dG, dB, None, ws)
    gamma, w = gamma.float().double(), w.float().double()
    h = 1e-5
    for t, got in ((x, dX), (gamma, dG), (beta, dB)):
        flat, out = t.view(-1), got.double().cpu().view(-1)
        for i in range(flat.numel()):
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss(x, gamma, beta)
            flat[i] = keep - h
            dn = loss(x, gamma, beta)
            flat[i] = keep
            assert abs((up - dn) / (2 * h) - float(out[i])) < 2e-5, i    # 64 u times values of order one


def test_rows_with_an_offset_keep_their_digits():
    """Features around 10000 with a spread of one: the deviations are exact in
    float32, so y is as good as the mean allows (64 u a = 0.04 of a step here)."""
    M, d = 64, 768
    X, g = make(M, d, F32, 3, offset=10000.0)
    Y = torch.empty(M, d, device=DEV)
    aa.aa_layernorm_fwd(X, None, None, Y)
    x, m, r, xh, _, _ = reference(X, None, None, 1e-5)
    a = x.abs().mean(1, keepdim=True)
    close(Y, xh, r * 64 * U * (a + (x - m).abs()) + 65 * U * xh.abs(), "offset rows")


def test_constant_rows_and_eps():
    X = torch.full((3, 40), 2.5, device=DEV)
    beta = torch.arange(40.0, device=DEV)
    Y, mean, rstd = torch.empty_like(X), torch.empty(3, device=DEV), torch.empty(3, device=DEV)
    aa.aa_layernorm_fwd(X, None, beta, Y, mean=mean, rstd=rstd, eps=0.25)
    assert torch.equal(Y, beta.expand(3, 40)) and bool((rstd == 2.0).all()) and bool((mean == 2.5).all())
    aa.aa_layernorm_fwd(X, None, beta, Y, eps=0.0)              # 0 * inf, as the formula has it
    assert bool(Y.isnan().all())


def test_a_row_of_nan_or_infinity_stays_alone():
    X, g = make(9, 300, F32, 4)
    Y0, Y1 = torch.empty_like(X), torch.empty_like(X)
    aa.aa_layernorm_fwd(X, None, None, Y0)
    X[4, 17], X[6, 2] = float("nan"), float("inf")
    aa.aa_layernorm_fwd(X, None, None, Y1)
    rest = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(Y0[rest], Y1[rest]) and bool(Y1[[4, 6]].isnan().all())


@pytest.mark.parametrize("xt,yt,dyt", [(BF16, BF16, BF16), (F32, F32, BF16), (BF16, F32, F32)])
def test_odd_rows_past_the_caches_equal_their_parts(xt, yt, dyt):
    """Rows of an odd width whose outputs go past the caches (more than 32 MB)
    start at any element address: the same bits as in calls of a few rows, which
    stay in the caches."""
    M, d, part = 16390, 1031, 745
    X, g = make(M, d, xt, 77)
    gamma, beta, D, dY = rand(g, (d,), F32), rand(g, (d,), F32), rand(g, (M, d), xt), rand(g, (M, d), dyt)
    S, dX = torch.empty_like(X), torch.empty_like(X)
    Y, mean, rstd = torch.empty(M, d, dtype=yt, device=DEV), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    assert min(t.numel() * t.element_size() for t in (Y, dX)) > 1 << 25
    aa.aa_layernorm_fwd(X, gamma, beta, Y, D, S, mean, rstd)
    aa.aa_layernorm_bwd(S, dY, gamma, mean, rstd, dX, dS=X)
    for lo in range(0, M, part):
        rows = slice(lo, min(lo + part, M))
        x, delta, s, dy, m, r = (t[rows].clone() for t in (X, D, S, dY, mean, rstd))
        s2, y, dx, m2, r2 = torch.empty_like(s), torch.empty_like(Y[rows]), torch.empty_like(x), *map(torch.empty_like, (m, r))
        aa.aa_layernorm_fwd(x, gamma, beta, y, delta, s2, m2, r2)
        aa.aa_layernorm_bwd(s, dy, gamma, m, r, dx, dS=x)
        assert all(torch.equal(a, b) for a, b in ((s2, s), (y, Y[rows]), (m2, m), (r2, r), (dx, dX[rows]))), lo


def test_in_place_forms_equal_the_others():
    M, d = 70, 1030
    X, g = make(M, d, BF16, 6)
    D, gamma = rand(g, (M, d), F32), rand(g, (d,), F32)
    S, Y, Y2 = torch.empty_like(X), torch.empty_like(X), torch.empty_like(X)
    aa.aa_layernorm_fwd(X, gamma, None, Y, D, S)
    X2 = X.clone()
    aa.aa_layernorm_fwd(X2, gamma, None, Y2, D, X2)
    assert torch.equal(S, X2) and torch.equal(Y, Y2)
    mean, rstd = torch.zeros(M, device=DEV), torch.ones(M, device=DEV)
    dS, dY = rand(g, (M, d), BF16), rand(g, (M, d), BF16)
    dX = torch.empty_like(dS)
    aa.aa_layernorm_bwd(X, dY, gamma, mean, rstd, dX, dS=dS)
    aa.aa_layernorm_bwd(X, dY, gamma, mean, rstd, dS, dS=dS)
    assert torch.equal(dX, dS)


def test_single_gradients_and_no_rows():
    M, d = 50, 130
    X, g = make(M, d, F32, 8)
    dY, mean, rstd = rand(g, (M, d), F32), torch.zeros(M, device=DEV), torch.ones(M, device=DEV)
    ws = torch.empty(aa.aa_layernorm_bwd_workspace(M, d), dtype=torch.uint8, device=DEV)
    dX, dG, dB = torch.empty_like(X), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    aa.aa_layernorm_bwd(X, dY, None, mean, rstd, dX, dG, dB, None, ws)
    for one in ("dgamma", "dbeta"):
        out = torch.full((d,), 5.0, device=DEV)
        aa.aa_layernorm_bwd(X, dY, None, mean, rstd, dX, workspace=ws, **{one: out})
        assert torch.equal(out, dG if one == "dgamma" else dB)
    # no rows: nothing is normalised, the sums are zero
    e = torch.empty(0, d, device=DEV)
    z = torch.empty(0, device=DEV)
    aa.aa_layernorm_fwd(e, None, None, torch.empty_like(e))
    aa.aa_layernorm_bwd(e, e, None, z, z, torch.empty_like(e), dG, dB)
    assert bool((dG == 0).all()) and bool((dB == 0).all())


def test_repeats_streams_and_graphs():
    """The same bits on every run, on another stream, and from two captured
    graphs that share a workspace, replayed in turn between eager calls."""
    M, d = 3000, 768
    X, g = make(M, d, F32, 9)
    gamma, dY = rand(g, (d,), F32), rand(g, (M, d), BF16)
    mean, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    ws = torch.empty(aa.aa_layernorm_bwd_workspace(M, d), dtype=torch.uint8, device=DEV)

    def call(x, y, dx, dg, db, stream=None):
        aa.aa_layernorm_fwd(x, gamma, None, y, mean=mean, rstd=rstd, stream=stream)
        aa.aa_layernorm_bwd(x, dY, gamma, mean, rstd, dx, dg, db, None, ws, stream=stream)

    def outs():
        return (torch.empty(M, d, dtype=BF16, device=DEV), torch.empty(M, d, device=DEV),
                torch.empty(d, device=DEV), torch.empty(d, device=DEV))

    X2 = X * 1.5 + 0.25
    ref, ref2 = outs(), outs()
    call(X, *ref)
    call(X2, *ref2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = outs()
    call(X, *o, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, ref))
    go, go2 = outs(), outs()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        call(X, *go)
    with torch.cuda.graph(g2):
        call(X2, *go2)
    for _ in range(4):
        for t in go + go2:
            t.zero_()
        g1.replay()
        g2.replay()
        call(X, *o)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(go, ref))
        assert all(torch.equal(a, b) for a, b in zip(go2, ref2))
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows equal those of a call of their own
    (a row does not depend on the others), rows of zeros add nothing."""
    d, k = 16384, 3
    M = (1 << 31) // d + 200
    X, dY = (torch.zeros(M, d, dtype=BF16, device=DEV) for _ in range(2))
    X[-k:], g = make(k, d, BF16, 12)
    dY[-k:] = rand(g, (k, d), BF16)
    gamma = rand(g, (d,), F32)
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    mean, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    dG, dB = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(aa.aa_layernorm_bwd_workspace(M, d), dtype=torch.uint8, device=DEV)
    aa.aa_layernorm_fwd(X, gamma, None, Y, mean=mean, rstd=rstd)
    aa.aa_layernorm_bwd(X, dY, gamma, mean, rstd, dX, dG, dB, None, ws)
    x, dy = X[-k:].clone(), dY[-k:].clone()
    y, dx, m, r = torch.empty_like(x), torch.empty_like(x), torch.empty(k, device=DEV), torch.empty(k, device=DEV)
    aa.aa_layernorm_fwd(x, gamma, None, y, mean=m, rstd=r)
    aa.aa_layernorm_bwd(x, dy, gamma, m, r, dx)
    assert torch.equal(Y[-k:], y) and torch.equal(dX[-k:], dx) and torch.equal(mean[-k:], m)
    assert torch.equal(rstd[-k:], r) and not bool(Y[:-k].any()) and not bool(dX[:-k].any())
    # k terms, each two roundings (the deviation and its product with rstd) and one of the product
    xh = (x.double() - m.double()[:, None]) * r.double()[:, None]
    mag = (dy.double() * xh).abs().sum(0) + (dy.double().abs() * (x.double().abs() + m.double().abs()[:, None]) *
                                             r.double()[:, None]).sum(0)
    close(dG, (dy.double() * xh).sum(0).cpu(), ((k + 3) * U * mag).cpu(), "dgamma")
    close(dB, dy.double().sum(0).cpu(), (k * U * dy.double().abs().sum(0)).cpu(), "dbeta")


def test_binding_refuses_before_the_library():
    X, Y = torch.zeros(4, 8, device=DEV), torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        aa.aa_layernorm_fwd(torch.zeros(8, 4, device=DEV).t(), None, None, Y)
    with pytest.raises(ValueError, match="shape"):
        aa.aa_layernorm_fwd(X, None, None, torch.zeros(4, 9, device=DEV))
    with pytest.raises(TypeError, match="dtype"):
        aa.aa_layernorm_fwd(X, torch.ones(8, device=DEV, dtype=BF16), None, Y)
    with pytest.raises(ValueError, match="on cpu"):
        aa.aa_layernorm_fwd(X, torch.ones(8), None, Y)
    with pytest.raises(aa.AAError, match="overlaps"):
        aa.aa_layernorm_fwd(X, None, None, X)
    with pytest.raises(aa.AAError, match="come together"):
        aa.aa_layernorm_fwd(X, None, None, Y, delta=X)
    with pytest.raises(aa.AAError, match="workspace"):
        aa.aa_layernorm_bwd(X, Y, None, torch.zeros(4, device=DEV), torch.zeros(4, device=DEV),
                            torch.zeros(4, 8, device=DEV), torch.zeros(8, device=DEV))
