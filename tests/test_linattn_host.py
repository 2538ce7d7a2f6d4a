"""Host side of linear attention and layer norm, on the CPU: the 64-bit
references against autograd and differences, the C ABI's validation, and the
binding's refusals."""
import ctypes

import numpy as np
import pytest
import torch

import nonlinear_rnn_solve_newton_b200 as pr
from tests import linattn_ref as ref
from tests.test_binding_marshalling import fake  # noqa: F401  (fixture)


# ------------------------------------------------------------------ references
def _loss_inputs(rng, B=2, L=5, H=4, Hk=2, Hv=1, Dk=3, Dv=2):
    f = rng.standard_normal
    return dict(q=f((B, L, H, Dk)), k=f((B, L, Hk, Dk)), v=f((B, L, Hv, Dv)),
                log_decay=-rng.uniform(0.05, 1.0, H), s0=f((B, H, Dk, Dv)),
                lengths=np.array([L, L - 2])), f((B, L, H, Dv)), f((B, H, Dk, Dv))


def test_reference_gradient_matches_differences():
    rng = np.random.default_rng(5)
    x, do, ds = _loss_inputs(rng)

    def loss(**y):
        o, s = ref.scan(**y, scale=0.7)
        return (o * do).sum() + (s * ds).sum()

    got = ref.backward(x["q"], x["k"], x["v"], x["log_decay"], do, s0=x["s0"], ds=ds, scale=0.7,
                       lengths=x["lengths"])
    # the loss is at most cubic along one coordinate of q, k, v or s0 (linear in each):
    # central differences are exact up to rounding, 2^-52 |loss| / h per entry
    for name, g in zip(("q", "k", "v", "s0"), got):
        flat = np.empty(g.size)
        for i in range(g.size):
            for sign in (1, -1):
                y = {n: np.array(a) for n, a in x.items()}
                y[name].reshape(-1)[i] += sign * 0.5
                flat[i] = loss(**y) if sign == 1 else flat[i] - loss(**y)
        assert np.max(np.abs(flat.reshape(g.shape) - g)) <= 1e-11


def test_reference_norm_matches_autograd():
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.standard_normal((7, 11))).requires_grad_()
    w = torch.from_numpy(rng.standard_normal(11)).requires_grad_()
    b = torch.from_numpy(rng.standard_normal(11)).requires_grad_()
    dy = rng.standard_normal((7, 11))
    y = torch.nn.functional.layer_norm(x, (11,), w, b, 1e-5)
    y.backward(torch.from_numpy(dy))
    ry, mean, rstd = ref.layer_norm(x.detach().numpy(), w.detach().numpy(), b.detach().numpy())
    dx, dw, db = ref.layer_norm_backward(dy, x.detach().numpy(), mean, rstd, w.detach().numpy())
    for got, want in ((ry, y.detach()), (dx, x.grad), (dw, w.grad), (db, b.grad)):
        assert np.allclose(got, want.numpy(), rtol=0, atol=1e-12)


# ------------------------------------------------------------------ C ABI
def _desc(**over):
    d = dict(B=2, L=5, H=4, Hq=4, Hk=2, Hv=4, Dk=16, Dv=24, scale=1.0)
    d.update(over)
    dense = {n: d.pop(n + "_stride", None) for n in ("q", "k", "v", "do")}
    s = pr._LinAttn(**d)
    for n, st in dense.items():
        getattr(s, n + "_stride")[:] = st or [1024, 128, 24]
    return s


BAD_SIZES = [dict(B=-1), dict(L=-1), dict(H=0), dict(Hq=3), dict(Hk=0), dict(Hv=8), dict(Dk=12),
             dict(Dv=136), dict(Dk=0), dict(L=1 << 31), dict(scale=float("nan")),
             dict(scale=float("inf")), dict(B=1 << 29)]


def test_linattn_abi_validation():
    lib = pr.load()
    vp = ctypes.c_void_p
    p, ws, odd = vp(4096), vp(1 << 20), vp(4104)

    def scan(d, q=p, k=p, v=p, g=p, s0=None, n=None, o=p, s=p, w=ws, nb=1 << 30):
        return lib.pararnn_scan_linattn(ctypes.byref(d), q, k, v, g, s0, n, o, s, w, nb, None, None,
                                        None)

    def back(d, q=p, k=p, v=p, g=p, s0=None, do=p, ds=None, n=None, dq=p, dk=p, dv=p, ds0=p, w=ws,
             nb=1 << 40):
        return lib.pararnn_scan_linattn_backward(ctypes.byref(d), q, k, v, g, s0, do, ds, n, dq,
                                                 dk, dv, ds0, w, nb, None, None, None)

    for bad in BAD_SIZES:
        d = _desc(**bad)
        assert lib.pararnn_linattn_workspace_size(ctypes.byref(d), 0) == 0, bad
        assert scan(d) == 1 and back(d) == 1, bad
    assert lib.pararnn_linattn_workspace_size(None, 0) == 0
    d = _desc()
    assert lib.pararnn_linattn_workspace_size(ctypes.byref(d), 0) > 0
    shared = lib.pararnn_linattn_workspace_size(ctypes.byref(d), 1)
    assert shared > lib.pararnn_linattn_workspace_size(ctypes.byref(_desc(Hk=4)), 1)
    for name in ("q", "k", "v", "g", "o"):
        assert scan(d, **{name: None}) == 1, name
    for name in ("q", "k", "v", "o", "s0", "s"):
        assert scan(d, **{name: odd}) == 1, name
    assert scan(d, g=vp(4097)) == 1 and scan(d, n=vp(4098)) == 1
    for name in ("q", "k", "v"):
        for st in ([0, 128, 24], [1024, -8, 24], [1024, 128, 12]):
            assert scan(_desc(**{name + "_stride": st})) == 1, (name, st)
    assert back(_desc(do_stride=[1024, 128, 20])) == 1
    long = _desc(L=4096)                      # cut into spans: their states need room
    need = lib.pararnn_linattn_workspace_size(ctypes.byref(long), 0)
    assert need > 256
    assert scan(long, w=None) == 6 and scan(long, nb=need - 1) == 6 and scan(long, w=vp(4100)) == 6
    for name in ("q", "k", "v", "g", "do", "dq", "dk", "dv"):
        assert back(d, **{name: None}) == 1, name
    assert back(d, do=odd) == 1 and back(d, dq=odd) == 1 and back(d, ds0=odd) == 1
    assert back(d, ds=p, ds0=p) == 1            # the gradient would race with its input
    assert back(d, w=None) == 6 and back(d, nb=shared - 1) == 6
    assert scan(_desc(B=0)) == 0 and back(_desc(B=0)) == 0   # nothing to do

    step = lib.pararnn_step_linattn

    def one(d, q=p, dt=0, g=p, sp=None, o=p, sn=p):
        return step(ctypes.byref(d), q, p, p, dt, g, sp, o, sn, None)

    assert one(_desc()) == 1                      # more than one token
    d1 = _desc(L=1)
    assert one(d1, dt=2) == 1 and one(d1, q=None) == 1 and one(d1, g=None) == 1
    assert one(d1, sn=None) == 1 and one(d1, sn=odd) == 1 and one(d1, sp=odd) == 1
    assert one(d1, q=vp(4098)) == 1 and one(_desc(L=1, B=0)) == 0


def test_layer_norm_abi_validation():
    lib = pr.load()
    vp = ctypes.c_void_p
    p, ws = vp(4096), vp(1 << 20)

    def fwd(x=p, xt=0, sx=8, w=None, b=None, y=p, yt=0, mean=p, rstd=p, M=3, D=8, eps=1e-5):
        return lib.pararnn_layer_norm(x, xt, sx, w, b, y, yt, mean, rstd, M, D, eps, None)

    def bwd(dy=p, yt=0, sdy=8, x=p, xt=0, sx=8, w=None, mean=p, rstd=p, dx=p, dw=p, db=p, M=3, D=8,
            s=ws, nb=1 << 20):
        return lib.pararnn_layer_norm_backward(dy, yt, sdy, x, xt, sx, w, mean, rstd, dx, dw, db,
                                               M, D, s, nb, None)

    for bad in (dict(M=-1), dict(D=0), dict(D=-4), dict(xt=2), dict(x=None), dict(x=vp(4098)),
                dict(sx=-1), dict(mean=None), dict(rstd=vp(4097)), dict(w=vp(4098))):
        assert fwd(**bad) == 1, bad
        assert bwd(**bad) == 1, bad
    for bad in (dict(yt=5), dict(y=None), dict(b=vp(2)), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf"))):
        assert fwd(**bad) == 1, bad
    for bad in (dict(dy=None), dict(dx=None), dict(dw=None), dict(db=vp(4098)), dict(sdy=-8)):
        assert bwd(**bad) == 1, bad
    assert bwd(s=None) == 6 and bwd(nb=8) == 6 and bwd(s=vp(4100)) == 6
    assert fwd(M=0) == 0
    assert lib.pararnn_layer_norm_workspace_size(-1, 8) == 0
    assert lib.pararnn_layer_norm_workspace_size(5, 0) == 0
    assert lib.pararnn_layer_norm_workspace_size(5, 8) > 0


# ------------------------------------------------------------------ binding
B, L, H, Dk, Dv = 2, 5, 4, 16, 24
BF = torch.bfloat16


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


class _Dev(torch.Tensor):
    """A host tensor that says it is on a device (the stand-in library reads nothing)."""
    is_cuda = True


def dv(t):
    return t.as_subclass(_Dev)


def qkv(**over):
    t = dict(q=z(B, L, H, Dk), k=z(B, L, 2, Dk), v=z(B, L, H, Dv), log_decay=z(H, dtype=torch.float32))
    t.update(over)
    return [dv(x) for x in t.values()]


def test_linattn_and_norm_reach_their_c_functions(fake):  # noqa: F811
    f32 = torch.float32
    st = z(B, H, Dk, Dv, dtype=f32)
    pack = z(B, L, H * Dk + 2 * Dk + H * Dv)
    q, k, v = pack.split([H * Dk, 2 * Dk, H * Dv], -1)
    views = [dv(q.unflatten(-1, (H, Dk))), dv(k.unflatten(-1, (2, Dk))),
             dv(v.unflatten(-1, (H, Dv)))]
    g = z(H, dtype=f32)
    x = dv(z(6, 8, dtype=f32))
    cases = [
        ("pararnn_scan_linattn", lambda: pr.scan_linattn(*qkv(), s0=st, lengths=z(
            B, dtype=torch.int32), state_out=st)),
        ("pararnn_scan_linattn", lambda: pr.scan_linattn(*views, g)),
        ("pararnn_scan_linattn_backward", lambda: pr.scan_linattn_backward(
            *views, g, dv(z(B, L, H, Dv)), s0=st, ds=st)),
        ("pararnn_step_linattn", lambda: pr.step_linattn(
            dv(z(B, H, Dk)), dv(z(B, 2, Dk)), dv(z(B, H, Dv)), g, st, state_out=st)),
        ("pararnn_layer_norm", lambda: pr.layer_norm(x, z(8, dtype=f32), out_dtype=BF)),
        ("pararnn_layer_norm", lambda: pr.layer_norm(dv(z(6, 3, 16))[..., :8])),
        ("pararnn_layer_norm_backward", lambda: pr.layer_norm_backward(
            x, x, z(6, dtype=f32), z(6, dtype=f32))),
    ]
    for name, call in cases:
        fake.calls.clear()
        call()
        assert [c for c in fake.calls if "workspace_size" not in c] == [name], name


def test_linattn_and_norm_refusals(fake):  # noqa: F811
    f32 = torch.float32
    st = z(B, H, Dk, Dv, dtype=f32)
    big = z(B * H * Dk * Dv + 8, dtype=f32)
    do = dv(z(B, L, H, Dv))
    x = dv(z(6, 8, dtype=f32))
    m = z(6, dtype=f32)
    bad = [
        lambda: pr.scan_linattn(*qkv(q=z(B, L, H, Dk, dtype=f32))),           # fp32 stream
        lambda: pr.scan_linattn(*qkv(k=z(B, L, 3, Dk))),                      # 3 does not divide 4
        lambda: pr.scan_linattn(*qkv(v=z(B, L + 1, H, Dv))),
        lambda: pr.scan_linattn(*qkv(q=z(B, L, H, 12), k=z(B, L, 2, 12))),    # 12 is no multiple of 8
        lambda: pr.scan_linattn(*qkv(v=z(B, L, H, 136))),
        lambda: pr.scan_linattn(*qkv(q=z(B, L, H, Dk * 2)[..., ::2])),        # strided last axis
        lambda: pr.scan_linattn(*qkv(q=z(B, L, H, Dk + 4)[..., :Dk])),        # stride 20
        lambda: pr.scan_linattn(*qkv(q=z(1, L, H, Dk).expand(B, L, H, Dk))),  # stride 0
        lambda: pr.scan_linattn(*qkv(q=z(B * L * H * Dk + 8)[4:-4].view(B, L, H, Dk))),
        lambda: pr.scan_linattn(*qkv(), s0=z(B, H, Dv, Dk, dtype=f32)),
        lambda: pr.scan_linattn(*qkv(), lengths=z(B, dtype=torch.int64)),
        lambda: pr.scan_linattn(*qkv(), out=z(B, L, H, Dv, dtype=f32)),
        lambda: pr.scan_linattn(*qkv(), s0=big[:-8].view(B, H, Dk, Dv),
                                state_out=big[8:].view(B, H, Dk, Dv)),        # partial overlap
        lambda: pr.scan_linattn(*qkv(log_decay=z(H))),                        # bf16 decays
        lambda: pr.scan_linattn_backward(*qkv(), dv(z(B, L, H, Dk))),
        lambda: pr.scan_linattn_backward(*qkv(), do, ds=st, out=(
            z(B, L, H, Dk), z(B, L, 2, Dk), z(B, L, H, Dv), st)),             # ds0 is ds
        lambda: pr.step_linattn(dv(z(B, H, Dk)), dv(z(B, 2, Dk, dtype=f32)), dv(z(B, H, Dv)),
                                z(H, dtype=f32)),                             # mixed types
        lambda: pr.step_linattn(*(dv(z(B, H, n, dtype=torch.float16)) for n in (Dk, Dk, Dv)),
                                z(H, dtype=f32)),
        lambda: pr.layer_norm(dv(z(6, 8, dtype=torch.float16))),
        lambda: pr.layer_norm(x, z(9, dtype=f32)),
        lambda: pr.layer_norm(dv(z(6, 0, dtype=f32))),
        lambda: pr.layer_norm(dv(z(8, 6, dtype=f32)).t()),                    # columns as rows
        lambda: pr.layer_norm(dv(z(4, 3, 10, 8, dtype=f32))[:, :, :5].transpose(0, 1)),
        lambda: pr.layer_norm(x, out_dtype=torch.float16),
        lambda: pr.layer_norm_backward(dv(z(5, 8, dtype=f32)), x, m, m),
        lambda: pr.layer_norm_backward(x, x, m, z(5, dtype=f32)),
    ]
    for i, call in enumerate(bad):
        fake.calls.clear()
        with pytest.raises((ValueError, TypeError)):
            call()
        assert [c for c in fake.calls if "workspace_size" not in c] == [], i


def test_linattn_and_norm_refuse_cpu_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        pr.scan_linattn(z(B, L, H, Dk), z(B, L, H, Dk), z(B, L, H, Dv), z(H, dtype=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        pr.step_linattn(z(B, H, Dk), z(B, H, Dk), z(B, H, Dv), z(H, dtype=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        pr.layer_norm(z(B, L))


def test_outputs_over_inputs_are_refused(fake):  # noqa: F811
    # the launches of a call read while others write: only a state may be its own output
    f32 = torch.float32
    q, k, v, g = qkv(k=z(B, L, H, Dk), v=z(B, L, H, Dk))
    do = dv(z(B, L, H, Dk))
    st, st2, m, w = (z(*s, dtype=f32) for s in ((B, H, Dk, Dk), (B, H, Dk, Dk), (6,), (8,)))
    x, dy = dv(z(6, 8, dtype=f32)), dv(z(6, 8, dtype=f32))
    q1, k1, v1 = (dv(z(B, H, Dk)) for _ in range(3))
    grads = [z(B, L, H, Dk) for _ in range(3)]
    bad = [
        lambda: pr.scan_linattn(q, k, v, g, out=v),
        lambda: pr.scan_linattn(q, k, v, g, out=q),
        lambda: pr.scan_linattn(q, k, v, g, s0=st, out=k, state_out=st),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, out=(q, *grads[1:], st)),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, out=(grads[0], grads[1], do, st)),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, out=(grads[0], grads[1], grads[1], st)),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, s0=st, out=(*grads, st)),
        lambda: pr.step_linattn(q1, k1, v1, g, out=v1),
        lambda: pr.step_linattn(q1, k1, v1, g, st, out=q1, state_out=st),
        lambda: pr.layer_norm(x, w, out=x),
        lambda: pr.layer_norm(x, w, stats=(m, m)),
        lambda: pr.layer_norm_backward(dy, x, m, z(6, dtype=f32), out=(dy, w, z(8, dtype=f32))),
        lambda: pr.layer_norm_backward(dy, x, m, z(6, dtype=f32), out=(x, w, z(8, dtype=f32))),
        lambda: pr.layer_norm_backward(dy, x, m, z(6, dtype=f32), out=(z(6, 8, dtype=f32), w, w)),
        lambda: pr.layer_norm_backward(dy, x, m, z(6, dtype=f32), w,
                                       out=(z(6, 8, dtype=f32), w, z(8, dtype=f32))),
    ]
    for i, call in enumerate(bad):
        fake.calls.clear()
        with pytest.raises(ValueError, match="overlap"):
            call()
        assert [c for c in fake.calls if "workspace_size" not in c] == [], i
    # neighbours in one allocation, and states updated in place, are fine
    buf = z(2 * B * L * H * Dk)
    near = buf.view(2, B, L, H, Dk)
    good = [
        lambda: pr.scan_linattn(dv(near[0]), k, v, g, s0=st, out=near[1], state_out=st),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, s0=st, ds=st, out=(*grads, st2)),
        lambda: pr.step_linattn(q1, k1, v1, g, st, state_out=st),
        lambda: pr.layer_norm(x, w, out=z(6, 8), stats=(m, z(6, dtype=f32))),
    ]
    for call in good:
        call()


def test_step_refuses_negative_strides():
    lib = pr.load()
    p = ctypes.c_void_p(4096)
    for name in ("q", "k", "v"):
        for st in ([-8, 0, 8], [8, 0, -8]):
            d = _desc(L=1, **{name + "_stride": st})
            assert lib.pararnn_step_linattn(ctypes.byref(d), p, p, p, 0, p, None, p, p, None) == 1


def test_layer_norm_refuses_rows_beyond_its_counters():
    # a column index is an int and runs up to 1024 beyond the row before it is compared:
    # rows of nearly 2^31 columns would wrap to negative offsets
    lib = pr.load()
    p = ctypes.c_void_p(4096)
    for D in ((1 << 31) - 1, (1 << 31) - 512, (1 << 30) + 8):
        assert lib.pararnn_layer_norm_workspace_size(2, D) == 0
        assert lib.pararnn_layer_norm(p, 0, D, None, None, p, 0, p, p, 0, D, 1e-5, None) == 1
        assert lib.pararnn_layer_norm_backward(p, 0, D, p, 0, D, None, p, p, p, p, p, 0, D,
                                               None, 0, None) == 1
    assert lib.pararnn_layer_norm_workspace_size(2, 1 << 30) > 0
    assert lib.pararnn_layer_norm(p, 0, 8, None, None, p, 0, p, p, 0, 1 << 30, 1e-5, None) == 0


def test_outputs_over_lengths_and_status_are_refused(fake):  # noqa: F811
    # every launch of a scan reads the lengths, and its status word is cleared first and
    # written last: no output may lie over either, and the word over no input
    f32, i32 = torch.float32, torch.int32
    q, k, v, g = qkv(k=z(B, L, H, Dk), v=z(B, L, H, Dk))
    do, n = dv(z(B, L, H, Dk)), z(B, dtype=i32)
    st, st2 = (z(B, H, Dk, Dk, dtype=f32) for _ in range(2))
    out = z(B, L, H, Dk)
    grads = (*(z(B, L, H, Dk) for _ in range(3)), st2)

    def word(t, at=0, size=1):   # int32s that lie inside a tensor
        return t.view(-1).view(i32)[at:at + size]

    bad = [
        lambda: pr.scan_linattn(q, k, v, g, lengths=word(out, 6, B), out=out),
        lambda: pr.scan_linattn(q, k, v, g, st, lengths=word(st, 30, B), state_out=st),
        lambda: pr.scan_linattn(q, k, v, g, lengths=n, status=n[1:]),
        lambda: pr.scan_linattn(q, k, v, g, status=word(g, 2)),
        lambda: pr.scan_linattn(q, k, v, g, status=word(q, 9)),
        lambda: pr.scan_linattn(q, k, v, g, st, status=word(st, 100)),
        lambda: pr.scan_linattn(q, k, v, g, out=out, status=word(out, 3)),
        lambda: pr.scan_linattn(q, k, v, g, state_out=st, status=word(st, 3)),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, lengths=n, status=n[:1]),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, status=word(do, 5)),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, s0=st, status=word(st, 5)),
        lambda: pr.scan_linattn_backward(q, k, v, g, do, out=grads, status=word(st2, 5)),
    ]
    for i, call in enumerate(bad):
        fake.calls.clear()
        with pytest.raises(ValueError, match="overlap"):
            call()
        assert [c for c in fake.calls if "workspace_size" not in c] == [], i
    two = z(B + 1, dtype=i32)    # neighbours are fine
    pr.scan_linattn(q, k, v, g, st, lengths=two[:B], out=out, state_out=st, status=two[B:])
    pr.scan_linattn(q, k, v, g, lengths=two[:B], status=two[B:])
    pr.scan_linattn_backward(q, k, v, g, do, lengths=two[:B], out=grads, status=two[B:])


def test_status_words_off_their_alignment_are_refused():
    # the kernels set the word by an atomic, which faults at such an address
    lib = pr.load()
    vp = ctypes.c_void_p
    d, p, ws, odd = _desc(), vp(4096), vp(1 << 20), vp(4098)
    assert lib.pararnn_scan_linattn(ctypes.byref(d), p, p, p, p, None, None, p, p, ws, 1 << 40, odd,
                                    None, None) == 1
    assert lib.pararnn_scan_linattn_backward(ctypes.byref(d), p, p, p, p, None, p, None, None, p, p,
                                             p, p, ws, 1 << 40, odd, None, None) == 1
