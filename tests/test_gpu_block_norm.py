"""GPU parity of the norms around a block against the oracle in 64 bits.

Tolerances, derived (u = 2^-24, half a step of fp32).  A sum of squares of dim
terms is taken in at most dim / (8 threads) + 10 additions of non-negative terms:
relative error below (dim / 256 + 16) u, a quarter of that step more for the
root; rsqrtf is within 2 ulp and __expf within 2 + |g| ulp for |g| < 100.  So a
factor is off by at most e = (dim / 256 + 24) u, with |g| <= 8 and the few
products: h by 2 e of the sum of its terms' sizes, and x by the same again plus
the relative error of the norm's root, at most rms(dh) / rms(h).  The last
rounding is half a step of the output's type (2^-8 bf16, 2^-24 fp32).
"""

import numpy as np
import pytest
import torch

from oracle import block_norm as ON
from paged_kv_cache_append_gb300 import nk

pytestmark = pytest.mark.gpu
DEV = "cuda"


def normal(shape, seed, mul=1.0):
    return (mul * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def bounds(r, y, gate, w, p, scale, rscale, sigmoid, offset, eps, dim, wide):
    """(x, h, allowance of x, allowance of h)."""
    x, h = ON.residual_norm(r, y, gate, w, p, eps, offset, scale, rscale, sigmoid)
    e = (dim / 256 + 24) * 2.0 ** -24
    size = np.abs(rscale * r) + np.abs(h - rscale * r)
    dh = 2 * e * size
    ah = dh + (2.0 ** -24 if wide else 2.0 ** -8) * (np.abs(h) + dh)
    if w is None:
        return None, h, None, ah
    root = np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    rel = np.sqrt(np.mean(dh * dh, -1, keepdims=True)) / root + 2 * e
    dx = np.abs(w + offset) / root * (dh + np.abs(h) * rel) * 1.01
    return x, h, dx + 2.0 ** -8 * (np.abs(x) + dx), ah


def check(N, dim, y=True, gate=None, post=False, weight=True, sigmoid=False, wide=False, scale=1.0, rscale=1.0, offset=0.0,
          eps=1e-6, pad=0, seed=0, mul=1.0):
    row = lambda s, m=1.0: normal((N, dim + pad), seed + s, m)[:, :dim]  # noqa: E731
    r = (torch.randn((N, dim + pad), generator=torch.Generator().manual_seed(seed + 9)) * 2)[:, :dim]
    r = r if wide else r.to(torch.bfloat16)
    yy = row(1, mul) if y else None
    g = row(2) if gate == "token" else normal((dim,), seed + 2) if gate == "channel" else None
    w = normal((dim,), seed + 3) if weight else None
    p = normal((dim,), seed + 4) if post else None
    d = lambda t: None if t is None else torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV).copy_(t)  # noqa: E731,E501
    n = nk.ResidualNorm(d(w), d(p), eps, scale, rscale, offset, sigmoid)
    x, h = nk.residual_norm(d(yy), d(r), n, d(g))
    torch.cuda.synchronize()
    rx, rh, ax, ah = bounds(f64(r), f64(yy), f64(g), f64(w), f64(p), scale, rscale, sigmoid, offset, eps, dim, wide)
    assert h.dtype == r.dtype and np.all(np.abs(f64(h) - rh) <= ah), np.max(np.abs(f64(h) - rh) - ah)
    if weight:
        assert x.dtype == torch.bfloat16 and np.all(np.abs(f64(x) - rx) <= ax), np.max(np.abs(f64(x) - rx) - ax)
    else:
        assert x is None


@pytest.mark.parametrize("dim", [8, 16, 24, 64, 72, 200, 256, 264, 512, 768, 1000, 2560, 4096, 4104, 8192, 8200, 12296,
                                 16384])
@pytest.mark.parametrize("N", [1, 5])
def test_dims(dim, N):
    check(N, dim, gate="token", post=True, sigmoid=True)
    check(N, dim, wide=True, scale=0.5, rscale=2.0)


@pytest.mark.parametrize("N", [1, 2, 3, 31, 129, 1000, 4001])
def test_rows(N):
    check(N, 96, gate="channel", post=True)
    check(N, 640, gate="token")


@pytest.mark.parametrize("y", [False, True])
@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_forms(y, gate, post, weight, wide):
    if not y and (gate or post):
        return
    for sigmoid in (False, True):
        check(3, 328, y=y, gate=gate, post=post, weight=weight, wide=wide, sigmoid=sigmoid, scale=-0.7, rscale=1.3,
              offset=1.0, eps=1e-3)


def test_padded_rows():
    check(7, 104, gate="token", post=True, pad=24)
    check(7, 2048, gate="token", wide=True, pad=8)


@pytest.mark.parametrize("mul", [2.0 ** -20, 2.0 ** 20])
def test_magnitudes(mul):
    """The post norm takes any magnitude of the block's output, tiny ones through eps."""
    check(3, 512, post=True, mul=mul)


def test_three_dimensions_and_in_place():
    y, r, w = normal((2, 3, 64), 1).to(DEV), normal((2, 3, 64), 2).to(DEV), normal((64,), 3).to(DEV)
    n = nk.ResidualNorm(w)
    x, h = nk.residual_norm(y, r, n)
    y2, r2 = y.clone(), r.clone()
    got = nk.residual_norm(y2, r2, n, out=y2, residual_out=r2)
    torch.cuda.synchronize()
    assert got[0] is y2 and got[1] is r2 and torch.equal(y2, x) and torch.equal(r2, h)


def test_zero_rows_and_non_finite_values_stay_in_their_rows():
    y, r, w = torch.zeros(4, 256).bfloat16(), torch.zeros(4, 256).bfloat16(), normal((256,), 1).to(DEV)
    y[1, 7], r[2, 9] = float("nan"), float("inf")
    y[3] = normal((256,), 2)
    x, h = nk.residual_norm(y.to(DEV), r.to(DEV), nk.ResidualNorm(w, post_weight=w))
    torch.cuda.synchronize()
    assert not x[0].any() and not h[0].any() and torch.isnan(x[1]).all() and torch.isfinite(x[3]).all()
    assert torch.isinf(h[2, 9])


def test_saturated_gates():
    """exp of a large negative gate overflows: the gate is 0, of a large one 1."""
    y, r = normal((2, 64), 1), torch.zeros(2, 64).bfloat16()
    g = torch.tensor([[-3e38], [3e38]]).expand(2, 64).bfloat16()
    _, h = nk.residual_norm(y.to(DEV), r.to(DEV), nk.ResidualNorm(None, sigmoid_gate=True), gate=g.to(DEV).contiguous())
    torch.cuda.synchronize()
    assert not h[0].any() and torch.equal(h[1].cpu(), y[1])


def test_rows_behind_are_not_written():
    y, w = normal((9, 64), 1).to(DEV), normal((64,), 2).to(DEV)
    buf = torch.full((9, 72), 7.0, device=DEV).bfloat16()
    ro = torch.full((9, 80), 5.0, device=DEV).bfloat16()
    nk.residual_norm(y[:5], y[:5], nk.ResidualNorm(w), out=buf[:5, :64], residual_out=ro[:5, :64])
    torch.cuda.synchronize()
    assert (buf[5:] == 7).all() and (buf[:, 64:] == 7).all() and (ro[5:] == 5).all() and (ro[:, 64:] == 5).all()


def test_captured_and_on_a_given_stream():
    y, r, w = normal((33, 4096), 1).to(DEV), normal((33, 4096), 2).to(DEV), normal((4096,), 3).to(DEV)
    n = nk.ResidualNorm(w, post_weight=w, scale=0.3)
    want = nk.residual_norm(y, r, n, gate=y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = nk.residual_norm(y, r, n, gate=y, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out = [torch.empty_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nk.residual_norm(y, r, n, gate=y, out=out[0], residual_out=out[1])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("power,low", [(127, -170.0), (60, -120.0), (0, -80.0)])
def test_gates_far_below_zero_scale_large_values(power, low, wide):
    """A logistic gate that fp32 cannot hold by itself (from -88 on) times a value that makes an ordinary number of it.

    e^-|g| is the square of 2^z, z = |g| / 2 log2 e <= 123: z is off by 2 half steps (2^-24 z each), which 2^z takes times
    ln 2, and by 2 ulp (2^-23) of the exponential: 2 * (123 * ln 2 + 2) ulp = 175, and 8 for the products and the
    division, less than 2^-15.2; then half a step of the output."""
    n = 512
    g = torch.linspace(low, 0.0, n).bfloat16().repeat(2, 1)
    y = ((1 + torch.rand((2, n), generator=torch.Generator().manual_seed(3)) * 0.9) * 2.0 ** power).bfloat16()
    r = torch.zeros((2, n), dtype=torch.float32 if wide else torch.bfloat16)
    _, h = nk.residual_norm(y.to(DEV), r.to(DEV), nk.ResidualNorm(None, sigmoid_gate=True), gate=g.to(DEV))
    torch.cuda.synchronize()
    want = f64(y) / (1 + np.exp(-f64(g)))
    assert np.all(np.abs(f64(h) - want) <= (2.0 ** -15.2 + (0 if wide else 2.0 ** -8)) * want)
