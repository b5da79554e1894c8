"""eps of the norms between blocks, forward and in every gradient: rows whose
variance is of eps' size, where it changes every value, and rows of zeros, where
1 / sqrt(eps) multiplies all.  FP32 throughout, so that the tolerances, in units
of u = 2^-24, also bind the gradients of layer norms closely.

Tolerances: a mean of a row is off by 64 u of the mean of absolute values; with
v off by o after centring, the factor 1 / sqrt(..) is off by rho, o's root mean
square times that factor and 100 u (sum of squares, division, root), one number
for a row; norm(v) by o times the factor and rho of itself.  A gradient through
a norm, r (g - n mean(g n) - mean g), is off by what its parts are, rho of their
sizes and 220 u for its own sums and products.

That eps is held to its place is checked on the oracle: with another eps in one
of the two norms some value is outside the tolerance."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from oracle import block_ops
from _gpu import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = [(6, 8), (6, 512), (7, 2120), (5, 7168), (5, 8200), (5, 16384)]
EPS = [(1.0, 0.5), (1e-3, 1e-5), (1e-3, 2e-7)]  # the values' size, eps
mean = lambda t: t.mean(-1, keepdims=True)


def make(T, n, size, seed):
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)
    p = lambda: 1 + 0.3 * randn(n)
    c = dict(x=size * (randn(T, n) + 0.2), residual=size * (randn(T, n) - 0.1), post=p(), gate=size * p(), pre=p(),
             gh=randn(T, n), gy=randn(T, n))
    c["x"][0], c["x"][2], c["residual"][2], c["residual"][3] = 0, 0, 0, 0  # x, both, the residual
    return {k: v.cuda() for k, v in c.items()}


def norm(v, ev, layer, eps):
    """norm(v), what it may be off by where v is off by ev, 1 / sqrt(..) and the share that may be off by."""
    n, r = block_ops.norm(v, layer, eps)
    off = ev + (64 * U * mean(np.abs(v)) + mean(ev) + U * np.abs(v) if layer else 0.0)
    rho = np.sqrt(mean(off * off)) * r + 100 * U
    return n, off * r + np.abs(n) * rho, r, rho


def through(g, eg, v, layer, eps):
    """The gradient of v through norm(v), and what it may be off by where g is off by eg."""
    n, en, r, rho = norm(v, np.zeros_like(v), layer, eps)
    a, size = np.abs(g), np.abs(n)
    parts = a + size * mean(a * size) + (mean(a) if layer else 0)
    err = eg + size * mean(eg * size + a * en) + en * mean(a * size) + (mean(eg) if layer else 0)
    return block_ops._through(g, v, layer, eps), r * (err + (220 * U + rho) * parts)


def forward(c, layer, eps_post, eps_pre):
    """{name: (value, what it may be off by before FP32's last rounding)}"""
    n, en, _, _ = norm(c["x"], np.zeros_like(c["x"]), layer, eps_post)
    w = c["post"] * c["gate"]
    h = 0.75 * c["residual"] + w * n
    eh = np.abs(w) * (en + 4 * U * np.abs(n)) + 4 * U * np.abs(0.75 * c["residual"])
    y, ey, _, _ = norm(h, eh + U * np.abs(h), layer, eps_pre)
    return {"h": (h, eh), "y": (c["pre"] * y, np.abs(c["pre"]) * (ey + 4 * U * np.abs(y)))}


def gradients(c, h, layer, eps_post, eps_pre):
    zero = np.zeros_like(h)
    depth = (64 + h.shape[0]) * U  # of a sum over rows
    d, ed = through(c["gy"] * c["pre"], 2 * U * np.abs(c["gy"] * c["pre"]), h, layer, eps_pre)
    n, en, _, _ = norm(h, zero, layer, eps_pre)
    out = {"pre": ((c["gy"] * n).sum(0), (np.abs(c["gy"]) * en).sum(0) + depth * np.abs(c["gy"] * n).sum(0))}
    d, ed = d + c["gh"], ed + 2 * U * (np.abs(d) + np.abs(c["gh"]))
    out["residual"] = 0.75 * d, 0.75 * (ed + 2 * U * np.abs(d))
    n, en, _, _ = norm(c["x"], zero, layer, eps_post)
    u, eu = n * c["post"], np.abs(c["post"]) * (en + 2 * U * np.abs(n))
    out["gate"] = (d * u).sum(0), (ed * np.abs(u) + np.abs(d) * eu).sum(0) + depth * np.abs(d * u).sum(0)
    d, ed = d * c["gate"], np.abs(c["gate"]) * (ed + 2 * U * np.abs(d))
    out["post"] = (d * n).sum(0), (ed * np.abs(n) + np.abs(d) * en).sum(0) + depth * np.abs(d * n).sum(0)
    out["x"] = through(d * c["post"], np.abs(c["post"]) * (ed + 2 * U * np.abs(d)), c["x"], layer, eps_post)
    return out


def check(got, want, others):
    """got within the tolerances of want; every one of others is not, in some value."""
    limit = {k: err + 2 * U * (np.abs(value) + err) for k, (value, err) in want.items()}
    for k, t in got.items():
        over = np.abs(t.double().cpu().numpy() - want[k][0]) / np.maximum(limit[k], 1e-300)
        assert np.all(over <= 1), (k, float(over.max()))
    for other in others:
        assert any(np.any(np.abs(other[k][0] - want[k][0]) > 2 * limit[k]) for k in got)


@pytest.mark.parametrize("T,n", SIZES)
@pytest.mark.parametrize("size,eps", EPS)
@pytest.mark.parametrize("layer", [False, True])
def test_forward(T, n, size, eps, layer):
    require_gpu()
    c = make(T, n, size, n)
    h, y = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    b.fp8_norm_residual(c["x"], c["residual"], h, y, pre_weight=c["pre"], post_norm=True, post_weight=c["post"],
                        gate=c["gate"], residual_scale=0.75, kind=b.FP8G_NORM_LAYER if layer else b.FP8G_NORM_RMS, eps=eps)
    f = {k: v.double().cpu().numpy() for k, v in c.items()}
    check({"h": h, "y": y}, forward(f, layer, eps, eps), [forward(f, layer, 1.01 * eps, eps), forward(f, layer, eps, 1.01 * eps)])
    assert not bool(h[2].any() or y[2].any())  # a row of zeros is one after both norms


@pytest.mark.parametrize("T,n", SIZES)
@pytest.mark.parametrize("size,eps", EPS)
@pytest.mark.parametrize("layer", [False, True])
def test_gradients(T, n, size, eps, layer):
    require_gpu()
    c = make(T, n, size, n + 1)
    h = c["residual"]  # any values do: the gradients are those at the h that they are given
    like = lambda *s: torch.empty(*s, device="cuda")
    got = dict(x=like(T, n), residual=like(T, n), pre=like(n), post=like(n), gate=like(n))
    b.fp8_norm_residual_backward(c["gh"], c["gy"], c["x"], h, *got.values(), pre_weight=c["pre"], post_norm=True,
                                 post_weight=c["post"], gate=c["gate"], residual_scale=0.75,
                                 kind=b.FP8G_NORM_LAYER if layer else b.FP8G_NORM_RMS, eps=eps)
    f = {k: v.double().cpu().numpy() for k, v in c.items()}
    check(got, gradients(f, f["residual"], layer, eps, eps),
          [gradients(f, f["residual"], layer, 1.01 * eps, eps), gradients(f, f["residual"], layer, eps, 1.01 * eps)])
