"""Layer norm on the GPU against 64 bits (tests/linattn_ref.py).

Bounds.  A row's mean is a sum of D fp32 terms: its error is at most E =
2^-23 (D / 32 + 40) mean|x| (a warp adds at most D / 32 terms in a row per lane,
then a tree; larger rows split further).  (x - mean) then carries E besides its
own rounding, the variance twice that relative to the row's spread, and y is
bounded by (|xh| 2^-21 + E rstd) |w| + the rounding of y's type.  Sums over M
rows in the gradient are held to 2^-23 (M / 64 + 400) times the sum of absolute
values: no column is added up in one run of more than M / 64 + 300 terms.
"""
import numpy as np
import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nonlinear_rnn_solve_newton_b200 as m

    m.load()
    return m


def dev(x, dtype=F32):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def host(t):
    return t.double().cpu().numpy()


def half(t):
    return torch.finfo(t).eps / 2


def make(M, D, seed, tx):
    rng = np.random.default_rng([seed, M, D])
    x = rng.standard_normal((M, D)) * 2 + rng.standard_normal((M, 1)) * 3
    x = ref.bf16(x) if tx == BF else x.astype(np.float32).astype(float)
    w, b = (rng.standard_normal(D).astype(np.float32).astype(float) for _ in range(2))
    return x, w, b, rng


def check_forward(x, w, b, got, ty, eps=1e-5):
    y, mean, rstd = ref.layer_norm(x, w, b, eps)
    D = x.shape[-1]
    E = 2.0 ** -23 * (D / 32 + 40) * np.abs(x).mean(-1)
    assert (np.abs(host(got[1]) - mean) <= E + 1e-30).all()
    rel = np.abs(host(got[2]) / rstd - 1)
    assert (rel <= 2.0 ** -21 + 2.0 ** -23 * (D / 32 + 40) + (E * rstd) ** 2).all(), rel.max()
    xh = np.abs(x - mean[..., None]) * rstd[..., None]
    aw = 1 if w is None else np.abs(w)
    tol = (xh * (2.0 ** -21 + 2.0 ** -23 * (D / 32 + 40)) + (E * rstd)[..., None]) * aw \
        + 2.0 ** -22 * np.abs(y) + half(ty) * np.abs(y) + 1e-30
    err = np.abs(host(got[0]) - y)
    assert (err <= tol).all(), float((err / tol).max())


def check_backward(dy, x, mean, rstd, w, got, tx):
    dx, dw, db = ref.layer_norm_backward(dy, x, mean, rstd, w)
    M, D = x.shape[0], x.shape[-1]
    xh = np.abs(x - mean[..., None]) * rstd[..., None]
    g = np.abs(dy) * (1 if w is None else np.abs(w))
    size = rstd[..., None] * (g + g.mean(-1, keepdims=True) + xh * (g * xh).mean(-1, keepdims=True))
    # x - mean loses half a step of the larger of the two, once in xh and once in the mean
    off = 2.0 ** -23 * (np.abs(x) + np.abs(mean)[..., None]) * rstd[..., None]
    extra = rstd[..., None] * (off * (g * xh).mean(-1, keepdims=True)
                               + xh * (g * off).mean(-1, keepdims=True))
    tol = 2.0 ** -23 * (D / 32 + 60) * size + extra + half(tx) * np.abs(dx) + 1e-30
    err = np.abs(host(got[0]) - dx)
    assert (err <= tol).all(), float((err / tol).max())
    lead = tuple(range(x.ndim - 1))
    F = 2.0 ** -23 * (M / 64 + 400)
    ady = np.abs(dy)
    assert (np.abs(host(got[1]) - dw) <= F * (ady * xh).sum(lead) + (ady * off).sum(lead)).all()
    assert (np.abs(host(got[2]) - db) <= F * ady.sum(lead)).all()


SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (1000, 128), (77, 100), (64, 1000), (33, 1024), (9, 1536),
         (300, 2056), (17, 4096), (7, 8192), (3, 16384), (2, 20011), (5000, 16), (2049, 72)]


@pytest.mark.parametrize("ty", [F32, BF])
@pytest.mark.parametrize("tx", [F32, BF])
@pytest.mark.parametrize("size", SIZES)
def test_norm_and_gradient(pr, size, tx, ty):
    x, w, b, rng = make(*size, 21, tx)
    X, W = dev(x, tx), dev(w)
    got = pr.layer_norm(X, W, dev(b), out_dtype=ty)
    assert got[0].dtype == ty
    check_forward(x, w, b, got, ty)
    dy = rng.standard_normal(size)
    dy = ref.bf16(dy) if ty == BF else dy.astype(np.float32).astype(float)
    grads = pr.layer_norm_backward(dev(dy, ty), X, got[1], got[2], W)
    assert grads[0].dtype == tx
    check_backward(dy, x, host(got[1]), host(got[2]), w, grads, tx)
    again = pr.layer_norm_backward(dev(dy, ty), X, got[1], got[2], W)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


@pytest.mark.parametrize("D", [64, 96, 100, 1000])
def test_views_without_weights(pr, D):
    """Row strides, odd offsets, leading axes, no weight and no bias."""
    x, _, _, rng = make(60, D, 22, F32)
    wide = torch.zeros(60, D + 9, device="cuda")
    for off in (0, 1, 4, 9):
        wide.zero_()
        wide[:, off:off + D] = dev(x)
        view = wide[:, off:off + D].unflatten(0, (5, 12))
        got = pr.layer_norm(view, eps=0.1)
        assert got[0].shape == (5, 12, D) and got[1].shape == (5, 12)
        check_forward(x.reshape(5, 12, D), None, None, got, F32, 0.1)
        dy = rng.standard_normal((60, D)).astype(np.float32).astype(float)
        wdy = torch.zeros(60, D + 3, device="cuda")
        wdy[:, 3:] = dev(dy)
        grads = pr.layer_norm_backward(wdy[:, 3:].unflatten(0, (5, 12)), view, got[1], got[2])
        flat = [grads[0].reshape(60, D), grads[1], grads[2]]
        check_backward(dy, x, host(got[1]).reshape(60), host(got[2]).reshape(60), None, flat, F32)


def test_constant_rows_and_large_means(pr):
    x = np.full((4, 640), 1000.0)
    x[1] += np.arange(640) % 2           # spread 0.5 about a mean of 1000.5
    x[2] = 0.0
    y, mean, rstd = pr.layer_norm(dev(x), eps=1e-5)
    ry, rm, rr = ref.layer_norm(x)
    assert torch.equal(y[0], torch.zeros(640, device="cuda")) and float(y[2].abs().max()) == 0
    assert np.abs(host(y)[1] - ry[1]).max() <= 1e-3  # mean 1000.5 is exact to 2^-14, spread 0.5
    assert np.allclose(host(rstd), rr, rtol=1e-3)


def test_non_finite_rows_stay_alone(pr):
    x, w, b, _ = make(9, 256, 23, F32)
    X = dev(x)
    X[4, 7], X[6, 0] = float("nan"), float("inf")
    y, mean, rstd = pr.layer_norm(X, dev(w), dev(b))
    bad = torch.zeros(9, dtype=torch.bool, device="cuda")
    bad[4] = bad[6] = True
    assert torch.equal(y.isnan().any(-1), bad)
    keep = [i for i in range(9) if i not in (4, 6)]
    check_forward(x[keep], w, b, (y[keep], mean[keep], rstd[keep]), F32)


def test_empty(pr):
    e = torch.empty(0, 48, device="cuda")
    y, mean, rstd = pr.layer_norm(e)
    assert y.shape == (0, 48) and mean.shape == (0,)
    dx, dw, db = pr.layer_norm_backward(e, e, mean, rstd)
    assert dx.shape == (0, 48) and float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


def test_gradient_against_differences(pr):
    """64-bit central differences of the formula's forward (truncation h^2 f''' / 6)."""
    x, w, b, rng = make(4, 24, 24, F32)
    dy = rng.standard_normal((4, 24)).astype(np.float32).astype(float)
    y, mean, rstd = pr.layer_norm(dev(x), dev(w), dev(b))
    dx, dw, db = pr.layer_norm_backward(dev(dy), dev(x), mean, rstd, dev(w))

    def loss(x, w, b):
        return (ref.layer_norm(x, w, b)[0] * dy).sum()

    for name, arr, got in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        got = host(got).reshape(-1)
        for i in range(0, got.size, 5):
            lo, hi = (dict(x=x.copy(), w=w.copy(), b=b.copy()) for _ in "ab")
            lo[name].reshape(-1)[i] -= 1e-4
            hi[name].reshape(-1)[i] += 1e-4
            want = (loss(**hi) - loss(**lo)) / 2e-4
            assert abs(got[i] - want) <= 1e-5 * (1 + np.abs(dy).sum())


def test_streams_and_graph(pr):
    x, w, b, rng = make(700, 384, 25, F32)
    X, W, Bb, dy = dev(x), dev(w), dev(b), dev(rng.standard_normal((700, 384)))

    def run(stream=None):
        y, mean, rstd = pr.layer_norm(X, W, Bb, stream=stream)
        return (y, mean, rstd, *pr.layer_norm_backward(dy, X, mean, rstd, W, stream=stream))

    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, outs))


@pytest.mark.parametrize("ty", [F32, BF])
@pytest.mark.parametrize("tx", [F32, BF])
@pytest.mark.parametrize("D,off", [(8193, 0), (16392, 0), (20011, 0), (8200, 1)])
def test_one_row_longer_than_registers(pr, D, off, tx, ty):
    """One row needs no workspace, however long: its sums go straight to the results."""
    x, w, b, rng = make(1, D, 26, tx)
    assert pr.load().pararnn_layer_norm_workspace_size(1, D) == 256
    wide = torch.zeros(1, D + off, dtype=tx, device="cuda")
    X = wide[:, off:]                    # off = 1: not on 16 bytes, an element an access
    X.copy_(dev(x, tx))
    got = pr.layer_norm(X, dev(w), dev(b), out_dtype=ty)
    check_forward(x, w, b, got, ty)
    dy = rng.standard_normal((1, D))
    dy = ref.bf16(dy) if ty == BF else dy.astype(np.float32).astype(float)
    grads = pr.layer_norm_backward(dev(dy, ty), X, got[1], got[2], dev(w))
    check_backward(dy, x, host(got[1]), host(got[2]), w, grads, tx)


@pytest.mark.parametrize("size", [(100000, 1), (70000, 8), (40000, 3)])
def test_many_short_rows(pr, size):
    x, w, b, rng = make(*size, 28, F32)
    if size[1] == 1:
        x = x * 0 + 0.5                  # a row of one is its own mean: y is the bias
    got = pr.layer_norm(dev(x), dev(w), dev(b))
    check_forward(x, w, b, got, F32)
    dy = rng.standard_normal(size).astype(np.float32).astype(float)
    grads = pr.layer_norm_backward(dev(dy), dev(x), got[1], got[2], dev(w))
    check_backward(dy, x, host(got[1]), host(got[2]), w, grads, F32)
