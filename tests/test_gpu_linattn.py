"""Linear attention with one decay per head on the GPU against the 64-bit
recurrence (tests/linattn_ref.py), through the binding.

Bounds.  Let A be the same recurrence on absolute values (every term of a sum
counted with its size).  The inputs are bf16 values both sides read exactly.
 * o (bf16): the output's own rounding is at most 2^-8 |o|.  The chunked form
   rounds two operands of its products to bf16, the weighted scores of the
   tokens of a chunk and the state at its start; a term of o passes through one
   of the two, so they add at most 2^-8 A.  fp32 sums add at most F A, with
   F = 2^-23 times the roundings a term can pass through: Dk + 2 x 128 in a
   chunk and 4 per chunk of 128 tokens (a token counts once in the recurrent
   form: at most L + Dk).
 * the state (fp32): F A (its products are exact to 2^-24 in both forms).
Besides, where an output has many entries, its error's 2-norm is held to what
independent roundings give: 2^-8 |o| (two roundings with rms 2^-8 / sqrt 3 make
0.82 of that) and 2^-18 |s| (random walks of up to 2^10 roundings of 2^-24).
"""
import numpy as np
import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pr():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nonlinear_rnn_solve_newton_b200 as m

    m.load()
    return m


def dev(x, dtype=torch.float32):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


BF = torch.bfloat16
DECAYS = [-np.inf, 0.0, -1e-4, -0.02, -0.4, -40.0]


def make(B, L, H, Hq, Hk, Hv, Dk, Dv, seed, state=True, lengths=None):
    rng = np.random.default_rng([seed, B, L, H, Dk, Dv])
    f = rng.standard_normal
    x = dict(q=ref.bf16(f((B, L, Hq, Dk))), k=ref.bf16(f((B, L, Hk, Dk))),
             v=ref.bf16(f((B, L, Hv, Dv))),
             log_decay=np.float32([DECAYS[(h + seed) % len(DECAYS)] for h in range(H)]).astype(float),
             s0=f((B, H, Dk, Dv)).astype(np.float32).astype(float) if state else None,
             lengths=None if lengths is None else np.asarray(lengths))
    y = dict(do=ref.bf16(f((B, L, H, Dv))),
             ds=f((B, H, Dk, Dv)).astype(np.float32).astype(float) if state else None)
    return x, y


def on_gpu(x):
    return dict(q=dev(x["q"], BF), k=dev(x["k"], BF), v=dev(x["v"], BF),
                log_decay=dev(x["log_decay"]), s0=dev(x["s0"]), lengths=dev(x["lengths"], torch.int32))


def absolute(x):
    return {n: (a if n in ("log_decay", "lengths") or a is None else np.abs(a))
            for n, a in x.items()}


def fp32_terms(L, Dk):
    return 2.0 ** -23 * max(Dk + 256 + 4 * (L // 128 + 2), L + Dk)


def check(got, want, size, f32, F, name):
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    tol = F * size + 1e-30 if f32 else 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + F) * size + 1e-30
    assert np.isfinite(got).all(), name
    assert (err <= tol).all(), (name, float(err.max()), float((err / tol).max()))
    if want.size >= 2000 and np.linalg.norm(want) > 0:
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= (2.0 ** -18 if f32 else 2.0 ** -8), (name, rel)


def check_scan(pr, x, scale, got):
    o, s = ref.scan(**x, scale=scale)
    ao, as_ = ref.scan(**absolute(x), scale=abs(scale))
    F = fp32_terms(x["q"].shape[1], x["q"].shape[-1])
    check(got[0], o, ao, False, F, "o")
    check(got[1], s, as_, True, F, "s")


def check_backward(pr, x, y, scale, got):
    want = ref.backward(**x, **y, scale=scale)
    size = ref.backward(**absolute(x), **absolute(y), scale=abs(scale))
    F = fp32_terms(x["q"].shape[1], 128)
    for g, w, a, n in zip(got, want, size, ("dq", "dk", "dv", "ds0")):
        check(g, w, a, n == "ds0", F, n)


# (B, L, H, Hq, Hk, Hv, Dk, Dv)
SHAPES = [(1, 1, 1, 1, 1, 1, 8, 8), (2, 2, 3, 3, 3, 3, 64, 64), (3, 15, 2, 2, 2, 2, 128, 128),
          (1, 16, 4, 4, 4, 4, 64, 128), (2, 17, 6, 2, 3, 6, 40, 24), (1, 127, 2, 2, 2, 2, 72, 64),
          (2, 128, 2, 1, 2, 2, 128, 64), (1, 129, 3, 3, 1, 3, 64, 96), (2, 300, 4, 4, 2, 1, 128, 128),
          (1, 777, 2, 2, 2, 2, 120, 8), (1, 1025, 1, 1, 1, 1, 128, 128)]


FORMS = {"auto": 0, "recurrent": 1, "chunks": 2}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
def test_scan(pr, shape, form):
    x, _ = make(*shape, seed=1)
    got = pr.scan_linattn(**on_gpu(x), scale=0.3, opts=pr.Options(regime=FORMS[form]))
    check_scan(pr, x, 0.3, got)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(pr, shape, form):
    x, y = make(*shape, seed=2)
    g = on_gpu(x)
    got = pr.scan_linattn_backward(**g, do=dev(y["do"], BF), ds=dev(y["ds"]), scale=0.3,
                                   opts=pr.Options(regime=FORMS[form]))
    check_backward(pr, x, y, 0.3, got)


def test_without_states(pr):
    x, y = make(2, 200, 3, 3, 3, 3, 64, 72, seed=3, state=False)
    g = on_gpu(x)
    check_scan(pr, x, 1.0, pr.scan_linattn(**g))
    check_backward(pr, x, y, 1.0, pr.scan_linattn_backward(**g, do=dev(y["do"], BF)))


@pytest.mark.parametrize("L,lengths", [(7, [7, 0, 3, 1]), (140, [139, 128, 0, 5]),
                                       (300, [-4, 300, 257, 1000])])
def test_padded_batch(pr, L, lengths):
    """Padding may hold anything; o's padded rows stay, gradients' are zero."""
    x, y = make(4, L, 3, 3, 3, 3, 64, 128, seed=4, lengths=lengths)
    g = on_gpu(x)
    do = dev(y["do"], BF)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), L)
        for t in (g["q"], g["k"], g["v"], do):
            t[b, n:] = float("nan")
            t[b, n + 1::2] = float("inf")
    out = torch.full((4, L, 3, 128), 7.5, dtype=BF, device="cuda")
    got = pr.scan_linattn(**g, scale=0.5, out=out)
    assert got[0] is out
    for b, n in enumerate(lengths):
        n = min(max(n, 0), L)
        assert (out[b, n:] == 7.5).all()
        out[b, n:] = 0
    check_scan(pr, x, 0.5, got)
    made = pr.scan_linattn(**g, scale=0.5)       # without out: padded rows are zero
    assert torch.equal(made[0], out) and torch.equal(made[1], got[1])
    check_backward(pr, x, y, 0.5,
                   pr.scan_linattn_backward(**g, do=do, ds=dev(y["ds"]), scale=0.5))


@pytest.mark.parametrize("L", [9, 210])
def test_strided_views(pr, L):
    """q, k, v as views of one packed projection; heads outside tokens; do a view."""
    B, H, Hk, Dk, Dv = 2, 4, 2, 64, 40
    x, y = make(B, L, H, H, Hk, H, Dk, Dv, seed=5)
    g = on_gpu(x)
    pack = torch.cat([g[n].flatten(2) for n in "qkv"], -1)
    assert not pack.isnan().any()
    q, k, v = pack.split([H * Dk, Hk * Dk, H * Dv], -1)
    views = dict(g, q=q.unflatten(-1, (H, Dk)), k=k.unflatten(-1, (Hk, Dk)),
                 v=v.unflatten(-1, (H, Dv)))
    heads_out = dict(g, **{n: g[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"})
    do = torch.zeros(B, L, H, Dv + 8, dtype=BF, device="cuda")
    do[..., :Dv] = dev(y["do"], BF)
    want = pr.scan_linattn(**g, scale=0.7)
    check_scan(pr, x, 0.7, want)
    grads = pr.scan_linattn_backward(**g, do=dev(y["do"], BF), ds=dev(y["ds"]), scale=0.7)
    for other in (views, heads_out):
        assert all(torch.equal(a, b) for a, b in zip(want, pr.scan_linattn(**other, scale=0.7)))
        again = pr.scan_linattn_backward(**other, do=do[..., :Dv], ds=dev(y["ds"]), scale=0.7)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_empty_calls(pr):
    H, Dk, Dv = 2, 16, 8
    for B, L in ((0, 5), (3, 0)):
        x, y = make(B, L, H, H, H, H, Dk, Dv, seed=6)
        g = on_gpu(x)
        o, s = pr.scan_linattn(**g)
        assert o.shape == (B, L, H, Dv) and torch.equal(s, g["s0"])
        dq, dk, dv, ds0 = pr.scan_linattn_backward(**g, do=dev(y["do"], BF), ds=dev(y["ds"]))
        assert dq.shape == g["q"].shape and torch.equal(ds0, dev(y["ds"]))
    g["s0"] = None
    assert (pr.scan_linattn(**g)[1] == 0).all()


def test_state_carried_over_pieces(pr):
    """A prompt scanned in pieces, the state updated in place, then single tokens."""
    x, _ = make(2, 300, 3, 3, 3, 3, 64, 64, seed=7)
    g = on_gpu(x)
    state = g["s0"].clone()
    outs = []
    for lo, hi in ((0, 131), (131, 290)):
        o, s = pr.scan_linattn(g["q"][:, lo:hi], g["k"][:, lo:hi], g["v"][:, lo:hi],
                               g["log_decay"], state, scale=0.2, state_out=state)
        assert s is state
        outs.append(o)
    for t in range(290, 300):
        o, s = pr.step_linattn(g["q"][:, t], g["k"][:, t], g["v"][:, t], g["log_decay"], state,
                               scale=0.2, state_out=state)
        assert s is state
        outs.append(o[:, None])
    check_scan(pr, x, 0.2, (torch.cat(outs, 1), state))


STEPS = [(1, 1, 1, 1, 1, 8, 8), (3, 4, 4, 2, 1, 128, 128), (70, 6, 3, 6, 6, 64, 96),
         (2, 5, 5, 5, 5, 72, 40), (33, 16, 16, 16, 16, 128, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("shape", STEPS)
def test_step(pr, shape, dtype):
    B, H, Hq, Hk, Hv, Dk, Dv = shape
    x, _ = make(B, 1, H, Hq, Hk, Hv, Dk, Dv, seed=8)
    g = on_gpu(x)
    q, k, v = (g[n][:, 0].to(dtype) for n in "qkv")
    o, s = pr.step_linattn(q, k, v, g["log_decay"], g["s0"], scale=1.5)
    assert o.dtype == dtype
    wo, ws = ref.scan(**x, scale=1.5)
    ao, as_ = ref.scan(**absolute(x), scale=1.5)
    F = 2.0 ** -23 * (Dk + 4)
    err = np.abs(o.double().cpu().numpy() - wo[:, 0])
    assert (err <= F * ao[:, 0] + (2.0 ** -8 * np.abs(wo[:, 0]) if dtype == BF else 0)).all()
    # gamma has two roundings of its own (expf and the product), the sum one
    assert (np.abs(s.double().cpu().numpy() - ws) <= 2.0 ** -22 * as_).all()
    assert torch.equal(pr.step_linattn(q, k, v, g["log_decay"], s0 := g["s0"].clone(), scale=1.5,
                                       state_out=s0)[1], s)
    zero = pr.step_linattn(q, k, v, g["log_decay"], scale=1.5)
    also = pr.step_linattn(q, k, v, g["log_decay"], torch.zeros_like(s), scale=1.5)
    assert all(torch.equal(a, b) for a, b in zip(zero, also))


def test_steps_equal_the_gradient_formula(pr):
    """Differences of the GPU's own forward: the loss is linear in each of s0, k's and
    v's entries, so a central difference has no truncation error, only rounding."""
    x, y = make(1, 40, 2, 2, 2, 2, 16, 16, seed=9)
    x["log_decay"] = np.array([-0.05, -0.3])
    g, do, ds = on_gpu(x), dev(y["do"], BF), dev(y["ds"])
    grads = pr.scan_linattn_backward(**g, do=do, ds=ds)

    def loss(h):
        o, s = ref.scan(**h)
        return (o * y["do"]).sum() + (s * y["ds"]).sum()

    rng = np.random.default_rng(1)
    size = ref.backward(**absolute(x), **absolute(y))
    for name, got, a in zip(("q", "k", "v", "s0"), grads, size):
        got = got.double().cpu().numpy().reshape(-1)
        for i in rng.integers(0, got.size, 12):
            lo, hi = ({n: (None if w is None else np.array(w)) for n, w in x.items()} for _ in "ab")
            lo[name].reshape(-1)[i] -= 0.5
            hi[name].reshape(-1)[i] += 0.5
            want = loss(hi) - loss(lo)
            assert abs(got[i] - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -7 * a.reshape(-1)[i]


def test_same_bits_every_call(pr):
    x, y = make(2, 900, 4, 4, 2, 4, 128, 128, seed=10)
    g, do, ds = on_gpu(x), dev(y["do"], BF), dev(y["ds"])
    one = (*pr.scan_linattn(**g), *pr.scan_linattn_backward(**g, do=do, ds=ds))
    for _ in range(3):
        two = (*pr.scan_linattn(**g), *pr.scan_linattn_backward(**g, do=do, ds=ds))
        assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_streams_and_graphs(pr):
    """Two calls at once on two streams, and two captured graphs replayed together."""
    xs = [make(1, 1500, 2, 2, 1, 2, 128, 64, seed=s) for s in (11, 12)]
    gs = [(on_gpu(x), dev(y["do"], BF), dev(y["ds"])) for x, y in xs]

    def run(i, stream=None):
        g, do, ds = gs[i]
        return (*pr.scan_linattn(**g, stream=stream),
                *pr.scan_linattn_backward(**g, do=do, ds=ds, stream=stream))

    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[run(i, streams[i]) for _ in range(3)][-1] for i in (0, 1)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graphs, outs = [], []
    for i in (0, 1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(i))
        graphs.append(graph)
    for o in outs:
        for t in o:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_status_word(pr):
    x, _ = make(1, 300, 2, 2, 2, 2, 64, 64, seed=13)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    pr.scan_linattn(**on_gpu(x), status=status)
    assert int(status) == 0


def test_layer_of_operators(pr):
    """norm -> projection -> linear attention -> norm of each head's rows and back, as a
    layer runs them, against the same layer in 64 bits on the values it rounds to."""
    B, L, H, D = 2, 140, 4, 256
    hd = D // H
    rng = np.random.default_rng(14)
    h = rng.standard_normal((B, L, D)).astype(np.float32)
    W = ref.bf16(rng.standard_normal((3 * D, D)) / 16)
    w, b = (rng.standard_normal(D).astype(np.float32) for _ in range(2))
    lam = np.float32([-0.5, -0.1, -0.02, 0.0])
    n, mean, rstd = pr.layer_norm(dev(h), dev(w), dev(b), out_dtype=BF)
    z = pr.input_projection(n, dev(W, BF), out_dtype=BF)
    q, k, v = (t.unflatten(-1, (H, hd)) for t in z.split([D, D, D], -1))
    o, s = pr.scan_linattn(q, k, v, dev(lam), scale=hd ** -0.5)
    y, ymean, yrstd = pr.layer_norm(o, out_dtype=torch.float32)
    dy = rng.standard_normal((B, L, H, hd)).astype(np.float32)
    do, _, _ = pr.layer_norm_backward(dev(dy), o, ymean, yrstd)
    dq, dk, dv_, _ = pr.scan_linattn_backward(q, k, v, dev(lam), do, scale=hd ** -0.5)
    torch.cuda.synchronize()

    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    rn, _, _ = ref.layer_norm(h, w, b)
    assert np.abs(f(n) - rn).max() <= 2.0 ** -8 * np.abs(rn).max() + 1e-5
    x = dict(q=f(q), k=f(k), v=f(v), log_decay=lam.astype(float), s0=None, lengths=None)
    check_scan(pr, x, hd ** -0.5, (o, s))
    ry, rm, rr = ref.layer_norm(f(o))
    # rstd is at most 1e5^(1/2) (eps) and xh at most sqrt(hd): 8 fp32 roundings of xh's size
    assert np.abs(f(y) - ry).max() <= 2.0 ** -20 * np.sqrt(hd)
    rdo, _, _ = ref.layer_norm_backward(dy, f(o), f(ymean), f(yrstd))
    assert np.linalg.norm(f(do) - rdo) <= 2.0 ** -8 * np.linalg.norm(rdo)
    check_backward(pr, x, dict(do=f(do), ds=None), hd ** -0.5,
                   (dq, dk, dv_, pr.scan_linattn_backward(q, k, v, dev(lam), do,
                                                          scale=hd ** -0.5)[3]))


@pytest.mark.parametrize("L", [100, 300, 2000])
@pytest.mark.parametrize("form", ["recurrent", "chunks"])
def test_non_finite_tokens_do_not_reach_back(pr, form, L):
    """A NaN or infinity in one token's k, v or q changes nothing before that token
    (gradients: nothing that does not depend on it), whatever chunk it lies in."""
    x, y = make(1, L, 3, 3, 3, 3, 64, 64, seed=15, state=False)
    x["log_decay"] = np.array([-0.01, -0.3, 0.0])
    opts = pr.Options(regime=FORMS[form])
    g, do = on_gpu(x), dev(y["do"], BF)
    clean = pr.scan_linattn(**g, opts=opts)
    t = L - 40
    for name, bad in (("v", float("nan")), ("k", float("inf")), ("v", float("-inf")), ("q", float("nan"))):
        h = {n: (a.clone() if n in "qkv" else a) for n, a in g.items()}
        h[name][0, t, 1, 5] = bad
        o, s = pr.scan_linattn(**h, opts=opts)
        # the chunked form walks such a head again in the recurrent form: other roundings
        assert torch.equal(o[:, :, ::2], clean[0][:, :, ::2])
        assert torch.equal(s[:, ::2], clean[1][:, ::2])
        assert o[:, :t].isfinite().all()
        bound = 2.0 ** -6 * clean[0].float().abs().max()
        assert (o[:, :t].float() - clean[0][:, :t].float()).abs().max() <= bound
        if name == "q":
            assert s.isfinite().all() and o[:, t + 1:].isfinite().all()
            assert not o[0, t, 1].isfinite().any()
        elif name == "v":
            assert not o[0, t:, 1, 5].isfinite().any() and not s[0, 1, :, 5].isfinite().any()
            keep = [i for i in range(64) if i != 5]
            assert o[0, t:, 1, keep].isfinite().all()
        else:
            assert not o[0, t:, 1].isfinite().any()
        # dq_t depends on k and v up to t, dv_t and dk_t on q and do from t on
        dq, dk, dv, ds0 = pr.scan_linattn_backward(**h, do=do, opts=opts)
        if name != "q":
            assert dq[0, :t].isfinite().all()
        else:
            assert dq.isfinite().all() and dk[0, t + 1:].isfinite().all()
            assert dv[0, t + 1:].isfinite().all()


def test_a_state_that_is_not_finite(pr):
    x, _ = make(1, 200, 2, 2, 2, 2, 64, 64, seed=16)
    x["log_decay"] = np.array([-0.1, -0.1])
    g = on_gpu(x)
    g["s0"][0, 1, 3, 7] = float("nan")
    before = g["s0"].clone()
    o, s = pr.scan_linattn(**g, state_out=g["s0"])  # in place: walked again from the old state
    keep = [i for i in range(64) if i != 7]
    assert o[0, :, 0].isfinite().all() and o[0, :, 1, keep].isfinite().all()
    assert o[0, :, 1, 7].isnan().all()
    again = pr.scan_linattn(**dict(g, s0=before))
    assert torch.equal(again[0].isnan(), o.isnan()) and torch.equal(again[1].isnan(), s.isnan())
    assert torch.equal(again[0].nan_to_num(), o.nan_to_num())


@pytest.mark.parametrize("L", [100, 300, 2000])
@pytest.mark.parametrize("form", ["recurrent", "chunks"])
@pytest.mark.parametrize("case", ["lowest", "large"])
def test_scores_beyond_fp32(pr, form, L, case):
    """Products q.k that overflow, though no output and no state does: a k of the type's
    lowest value whose v is zero, and large q and k whose v is small."""
    x, _ = make(1, L, 3, 3, 3, 3, 64, 64, seed=19, state=False)
    x["log_decay"] = np.array([-0.01, -0.3, 0.0])
    t = L - 40
    if case == "lowest":
        x["k"][0, t, 1] = float(torch.finfo(BF).min)
        x["v"][0, t, 1] = 0.0
    else:
        x["q"][0, t:, 1] *= 2.0 ** 80
        x["k"][0, t, 1] *= 2.0 ** 80
        x["v"][0, t, 1] *= 2.0 ** -90
    check_scan(pr, x, 0.25, pr.scan_linattn(**on_gpu(x), scale=0.25,
                                            opts=pr.Options(regime=FORMS[form])))


def test_many_steps_keep_the_state(pr):
    """Thousands of decode steps with slow decays: what each rounds must not add up in
    one direction.  A step rounds gamma s + k v twice (2^-24 each); over the 3000 steps of
    the walk independent roundings give at most 2^-24 (2 x 3000)^(1/2) = 2^-17.7 of the
    state's size, while the half step that gamma as one float leaves, 2^-25 a token, would
    be 3000 of them, 2^-13.4."""
    H, D, n = 6, 64, 3000
    rng = np.random.default_rng(20)
    lam = np.float32([-1e-4, -2.3e-4, -3.7e-5, -5.1e-4, -7e-5, -1.3e-5]).astype(float)
    s = rng.standard_normal((1, H, D, D)).astype(np.float32)
    want = s.astype(np.float64)
    k, v = (ref.bf16(rng.standard_normal((n, 1, H, D))) for _ in range(2))
    q = dev(k[0], BF)
    got, gk, gv, g = dev(s), dev(k, BF), dev(v, BF), dev(lam)
    gamma = np.exp(lam)[:, None, None]
    for t in range(n):
        pr.step_linattn(q, gk[t], gv[t], g, got, state_out=got)
        want = gamma * want + k[t][..., :, None] * v[t][..., None, :]
    for h in range(H):
        a, b = got[0, h].double().cpu().numpy(), want[0, h]
        assert np.linalg.norm(a - b) <= 2.0 ** -17 * np.linalg.norm(b), (
            h, np.linalg.norm(a - b) / np.linalg.norm(b))


def same_infinities(got, want, size, f32, F, name):
    """Non-finite entries are the reference's (NaN where it has NaN, infinities of its
    sign); the others stay within the bounds of `check`."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any(), name
    ok = np.isfinite(want)
    tol = F * size + 1e-30 if f32 else 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + F) * size + 1e-30
    assert (np.abs(got[ok] - want[ok]) <= tol[ok]).all(), name


def infinite(shape, rng):
    """fp32 states with one infinity of each sign in every head, in different columns."""
    s = rng.standard_normal(shape).astype(np.float32).astype(float)
    s[..., 3, 5], s[..., 1, 2] = np.inf, -np.inf
    return s


# gamma: 1, one float alone, two floats, below fp32, none
INF_DECAYS = np.float32([0.0, -0.4, -1e-3, -0.2, -200.0, -np.inf]).astype(float)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (72, 40), (8, 8)])
def test_step_keeps_infinite_states(pr, Dk, Dv, dtype):
    """gamma inf is inf, whatever gamma's parts (0 inf = NaN for gamma = 0 alone)."""
    H = len(INF_DECAYS)
    x, _ = make(2, 1, H, H, H, H, Dk, Dv, seed=27)
    x["log_decay"] = INF_DECAYS
    x["s0"] = infinite(x["s0"].shape, np.random.default_rng(27))
    x["v"][1, 0, :, 1] = np.inf             # and an infinite v: k v, in every row
    x["k"][1] = np.abs(x["k"][1])           # of one sign, so that the output is too
    x["q"][1] = np.abs(x["q"][1])
    g = on_gpu(x)
    o, s = pr.step_linattn(*(g[n][:, 0].to(dtype) for n in "qkv"), g["log_decay"], g["s0"])
    with np.errstate(invalid="ignore"):
        wo, ws = ref.scan(**x)
        ao, as_ = ref.scan(**absolute(x))
    assert np.isinf(ws).any() and np.isinf(wo).any()
    same_infinities(s, ws, as_, True, 2.0 ** -22, "s")
    same_infinities(o[:, None], wo, ao, dtype == torch.float32, 2.0 ** -23 * (Dk + 4), "o")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("L", [5, 200, 2100])
def test_scans_keep_infinite_states(pr, form, L):
    """Both forms, one span and several: an infinite state stays what the recurrence makes
    of it, to the end and in the gradients that meet it."""
    H = len(INF_DECAYS)
    x, y = make(1, L, H, H, H, H, 64, 72, seed=28)
    rng = np.random.default_rng(28)
    x["log_decay"] = INF_DECAYS
    x["s0"], y["ds"] = infinite(x["s0"].shape, rng), infinite(x["s0"].shape, rng)
    opts = pr.Options(regime=FORMS[form])
    F = fp32_terms(L, 128)
    with np.errstate(invalid="ignore"):
        want, size = ref.scan(**x, scale=0.3), ref.scan(**absolute(x), scale=0.3)
        grads = ref.backward(**x, **y, scale=0.3)
        gsize = ref.backward(**absolute(x), **absolute(y), scale=0.3)
    assert np.isinf(want[1]).any() and np.isinf(grads[3]).any()
    got = pr.scan_linattn(**on_gpu(x), scale=0.3, opts=opts)
    for a, w, z, n in zip(got, want, size, ("o", "s")):
        same_infinities(a, w, z, n == "s", F, n)
    got = pr.scan_linattn_backward(**on_gpu(x), do=dev(y["do"], BF), ds=dev(y["ds"]), scale=0.3,
                                   opts=opts)
    for a, w, z, n in zip(got, grads, gsize, ("dq", "dk", "dv", "ds0")):
        same_infinities(a, w, z, n == "ds0", F, n)


@pytest.mark.parametrize("form", ["recurrent", "chunks"])
def test_an_infinite_token_leaves_an_infinite_state(pr, form):
    """A v of one token is infinite: so is the state behind it, in its column alone, over
    the rest of the prompt and its spans."""
    x, _ = make(1, 2100, 2, 2, 2, 2, 64, 64, seed=29, state=False)
    x["log_decay"] = np.array([-0.01, 0.0])
    x["v"][0, 300, 1, 7] = np.inf
    with np.errstate(invalid="ignore"):
        want, size = ref.scan(**x), ref.scan(**absolute(x))
    assert np.isinf(want[1][0, 1, :, 7]).all()
    got = pr.scan_linattn(**on_gpu(x), opts=pr.Options(regime=FORMS[form]))
    for a, w, z, n in zip(got, want, size, ("o", "s")):
        same_infinities(a, w, z, n == "s", fp32_terms(2100, 64), n)


# Walks cut into spans of time: few heads, long rows.  (B, L, H, Hq, Hk, Hv, Dk, Dv) and the
# rows' lengths: whole, within the first span, nothing, at the end of a chunk (and with these
# sizes of a span), one token beyond.
SPANS = [((1, 2050, 2, 2, 2, 2, 64, 64), None),
         ((1, 2200, 3, 1, 3, 1, 128, 72), None),
         ((1, 2500, 2, 2, 1, 2, 72, 128), None),
         ((2, 1300, 1, 1, 1, 1, 128, 128), [640, 1300]),
         ((5, 2300, 2, 2, 1, 2, 64, 64), [2300, 100, 0, 1280, 1281]),
         ((3, 2300, 2, 1, 2, 2, 128, 72), [768, 2300, 2177]),
         ((4, 2304, 1, 1, 1, 1, 96, 112), [2304, 0, 384, 129])]


def spans_of(pr, g, do):
    """Spans of the forward walk and of the gradients', from the workspaces they ask for."""
    d = pr._linattn_desc(g["q"], g["k"], g["v"], g["log_decay"], 1.0, BF, do)
    state, rows = 4 * d.B * d.H * d.Dk * d.Dv, 4 * d.B * d.L * d.H
    shared = sum(-(-rows * n // 512) * 512 for n, h in ((d.Dk, d.Hq), (d.Dk, d.Hk), (d.Dv, d.Hv))
                 if h != d.H)
    lib = pr.load()
    return pr._linattn_ws(lib, d, 0) // state, (pr._linattn_ws(lib, d, 1) - shared) // (3 * state)


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("i", range(len(SPANS)))
def test_spans(pr, i, state):
    """Both directions over several spans against the recurrence: states carried over the
    join, lengths that end inside, before and between spans, heads that are shared."""
    shape, lengths = SPANS[i]
    for seed in (31 + i, 34 + i):            # other decays
        x, y = make(*shape, seed=seed, state=state, lengths=lengths)
        g, do = on_gpu(x), dev(y["do"], BF)
        assert min(spans_of(pr, g, do)) > 1
        B, L, H, Dv = shape[0], shape[1], shape[2], shape[7]
        for b, n in enumerate(lengths or ()):
            for t in (g["q"], g["k"], g["v"], do):
                t[b, n:] = float("nan")
                t[b, n + 1::2] = float("inf")
        out = torch.full((B, L, H, Dv), 7.5, dtype=BF, device="cuda")
        got = pr.scan_linattn(**g, scale=0.4, out=out)
        for b, n in enumerate(lengths or ()):
            assert (out[b, n:] == 7.5).all()
            out[b, n:] = 0
        check_scan(pr, x, 0.4, got)
        check_backward(pr, x, y, 0.4, pr.scan_linattn_backward(**g, do=do, ds=dev(y["ds"]), scale=0.4))
        if state:                            # the state in place: the join reads and writes it
            s = g["s0"].clone()
            again = pr.scan_linattn(**dict(g, s0=s), scale=0.4, state_out=s)
            assert again[1] is s and torch.equal(s, got[1]) and torch.equal(again[0], out)


def test_spans_of_strided_views(pr):
    B, L, H, Hk, Dk, Dv = 1, 2100, 4, 2, 64, 40
    x, y = make(B, L, H, H, Hk, H, Dk, Dv, seed=38)
    g, do = on_gpu(x), dev(y["do"], BF)
    assert min(spans_of(pr, g, do)) > 1
    pack = torch.cat([g[n].flatten(2) for n in "qkv"], -1)
    q, k, v = pack.split([H * Dk, Hk * Dk, H * Dv], -1)
    views = dict(g, q=q.unflatten(-1, (H, Dk)), k=k.unflatten(-1, (Hk, Dk)),
                 v=v.unflatten(-1, (H, Dv)))
    got = pr.scan_linattn(**views, scale=0.7)
    check_scan(pr, x, 0.7, got)
    assert all(torch.equal(a, b) for a, b in zip(got, pr.scan_linattn(**g, scale=0.7)))
    grads = pr.scan_linattn_backward(**views, do=do, ds=dev(y["ds"]), scale=0.7)
    check_backward(pr, x, y, 0.7, grads)


@pytest.mark.parametrize("L", [300, 2050])
def test_a_wait_that_ran_out_does_not_hold_the_gpu(pr, L):
    """Where a wait runs out, the CTA waits for the copies that it asked for and for no
    others: a call ends in far less than the two seconds that each such wait may take."""
    x, y = make(1, L, 2, 2, 1, 2, 128, 64, seed=39)
    g, do, ds = on_gpu(x), dev(y["do"], BF), dev(y["ds"])
    opts = pr.Options(regime=2, wait_timeout_ns=1)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    torch.cuda.synchronize()
    ends[0].record()
    pr.scan_linattn(**g, opts=opts)
    pr.scan_linattn_backward(**g, do=do, ds=ds, opts=opts)
    ends[1].record()
    torch.cuda.synchronize()
    assert ends[0].elapsed_time(ends[1]) < 1000


@pytest.mark.parametrize("L", [300, 2050])
def test_waits_that_run_out(pr, L):
    """Waits of a few microseconds end in the status word: where it says 0 the call has done all
    of its work.  A call after it is right.  One span, and several."""
    x, y = make(1, L, 2, 2, 1, 2, 128, 64, seed=39)
    g, do, ds = on_gpu(x), dev(y["do"], BF), dev(y["ds"])
    want = (*pr.scan_linattn(**g), *pr.scan_linattn_backward(**g, do=do, ds=ds))
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    for limit in (1, 2000, 4000, 8000, 16000) * 8:
        opts = pr.Options(regime=2, wait_timeout_ns=limit)
        got = pr.scan_linattn(**g, opts=opts, status=status[:1])
        got += pr.scan_linattn_backward(**g, do=do, ds=ds, opts=opts, status=status[1:])
        words = status.tolist()
        assert set(words) <= {0, 4}
        for w, a, b in ((words[0], want[:2], got[:2]), (words[1], want[2:], got[2:])):
            assert w == 4 or all(torch.equal(p, q) for p, q in zip(a, b))
    again = pr.scan_linattn(**g, status=status[:1])
    again += pr.scan_linattn_backward(**g, do=do, ds=ds, status=status[1:])
    assert status.tolist() == [0, 0]
    assert all(torch.equal(p, q) for p, q in zip(want, again))


@pytest.mark.parametrize("L", [6, 200, 2050])
def test_growing_heads(pr, L):
    """gamma above 1 (a positive log decay) within the range of fp32: one token at a time, one
    span and several.  The bounds go by the sums of sizes, which grow with the state."""
    x, y = make(1, L, 2, 2, 2, 2, 64, 64, seed=40)
    x["log_decay"] = np.float32([0.02, 0.001]).astype(float)
    g = on_gpu(x)
    check_scan(pr, x, 0.3, pr.scan_linattn(**g, scale=0.3))
    check_backward(pr, x, y, 0.3, pr.scan_linattn_backward(**g, do=dev(y["do"], BF),
                                                           ds=dev(y["ds"]), scale=0.3))


def test_one_tensor_as_several_streams(pr):
    x, y = make(2, 150, 3, 3, 3, 3, 64, 64, seed=41)
    x["k"] = x["v"] = x["q"]
    g = on_gpu(x)
    g["k"] = g["v"] = g["q"]
    check_scan(pr, x, 0.3, pr.scan_linattn(**g, scale=0.3))
    y["do"] = x["q"]
    check_backward(pr, x, y, 0.3, pr.scan_linattn_backward(**g, do=g["q"], ds=dev(y["ds"]), scale=0.3))
