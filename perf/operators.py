"""Measured cases of the linear-attention and layer-norm operators.

Two families: linear attention with one decay per head (the chunked scan over a
prompt, its gradients, the step for one token) and layer norm (forward, backward
with the weight's gradient).  ``run`` computes an operator in elementary torch
operations, or calls the package where ``own`` is true.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases
def _scan(name, op, B, L, H, Dk, Dv, Hk=0, Hv=0, packed=False, padded=False, state=False):
    c = {"op": op, "B": B, "L": L, "H": H, "Hk": Hk or H, "Hv": Hv or H, "Dk": Dk, "Dv": Dv,
         "packed": packed, "padded": padded, "state": state}
    return dict(c, name=name) if name else c


def _step(name, B, H, Dk, Dv, fp32=False, Hk=0):
    c = {"op": "step", "B": B, "H": H, "Hk": Hk or H, "Dk": Dk, "Dv": Dv, "fp32": fp32}
    return dict(c, name=name) if name else c


def _norm(name, op, M, D, x="f32", y="bf16"):
    c = {"op": op, "M": M, "D": D, "x": x, "y": y}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short prompt of one request: latency
        _scan("scan_one_prompt", "scan", 1, 37, 8, 64, 64, state=True),
        # the framework's middle workload (B=8, L=4096, D=1024) as 8 heads of 128
        _scan("scan_b8_l4096_d1024", "scan", 8, 4096, 8, 128, 128),
        # the language-model width (B=8, L=8192, D=4096) as 32 heads of 128
        _scan("scan_b8_l8192_d4096", "scan", 8, 8192, 32, 128, 128, state=True),
        # one long document: few heads, the work is split over time
        _scan("scan_b1_l65536_h12", "scan", 1, 65536, 12, 128, 64),
        # a padded batch of prompts, q/k shared by head groups, views of one projection
        _scan("scan_padded_packed", "scan", 6, 1531, 12, 64, 96, Hk=4, packed=True, padded=True,
              state=True),
        # a training step of the middle workload
        _scan("bwd_b8_l4096_d1024", "backward", 8, 4096, 8, 128, 128),
        # a ragged training batch with shared key and value heads and carried state
        _scan("bwd_shared_heads", "backward", 5, 1111, 9, 72, 128, Hk=3, Hv=3, padded=True,
              state=True),
        # decoding: one request, and a full serving batch
        _step("step_b1_h8", 1, 8, 128, 128),
        _step("step_b192_h32", 192, 32, 128, 128),
        # the fp32 solution of a layer to the bf16 input of the next projection
        _norm("norm_32768x1024", "norm", 32768, 1024),
        # per-head rows of the attention's output, in training
        _norm("norm_bwd_heads_262144x128", "norm_bwd", 262144, 128, x="bf16"),
        # the language-model width
        _norm("norm_bwd_16384x4096", "norm_bwd", 16384, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "backward", "step", "norm", "norm_bwd"])
    if op in ("scan", "backward"):
        while True:
            B, L, H = _log(rng, 1, 16), _log(rng, 1, 30000), _log(rng, 1, 64)
            Dk, Dv = (rng.choice([64, 128, 64, 128, 8 * rng.randint(1, 16)]) for _ in range(2))
            if B * L * H * max(Dk, Dv) <= (1 << 27):
                break
        parts = [d for d in range(1, H + 1) if H % d == 0]
        shared = rng.random() < 0.3
        return _scan(None, op, B, L, H, Dk, Dv, Hk=rng.choice(parts) if shared else H,
                     Hv=rng.choice(parts) if shared else H, packed=rng.random() < 0.4,
                     padded=rng.random() < 0.4, state=rng.random() < 0.5)
    if op == "step":
        B, H = _log(rng, 1, 256), _log(rng, 1, 48)
        Dk, Dv = (rng.choice([64, 128, 8 * rng.randint(1, 16)]) for _ in range(2))
        return _step(None, B, H, Dk, Dv, fp32=rng.random() < 0.4)
    while True:
        M, D = _log(rng, 1, 300000), _log(rng, 8, 16384)
        if rng.random() < 0.7:
            D = -(-D // 8) * 8
        if M * D <= (1 << 26):
            break
    return _norm(None, op, M, D, x=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]))


# --------------------------------------------------------------------------- inputs
def _decay(H, g):
    """One log decay per head, memories from a few tokens to a few thousand."""
    h = torch.arange(H, device=DEV, dtype=torch.float32)
    u = torch.rand(H, device=DEV, generator=g)
    return -torch.exp2(-1.0 - 9.0 * (h + u) / H)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, device=DEV, generator=g).to(dtype)

    if op in ("scan", "backward"):
        B, L, H, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "L", "H", "Hk", "Hv", "Dk", "Dv"))
        if case["packed"]:  # views of one projection's output
            z = rand(B, L, H * Dk + Hk * Dk + Hv * Dv)
            q, k, v = z.split([H * Dk, Hk * Dk, Hv * Dv], dim=-1)
            q, k, v = q.unflatten(-1, (H, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (Hv, Dv))
        else:
            q, k, v = rand(B, L, H, Dk), rand(B, L, Hk, Dk), rand(B, L, Hv, Dv)
        s = {"op": op, "q": q, "k": k, "v": v, "log_decay": _decay(H, g), "scale": Dk ** -0.5,
             "lengths": None, "s0": None}
        if case["padded"]:
            n = torch.randint(max(1, L // 2), L + 1, (B,), device=DEV, generator=g)
            s["lengths"] = n.to(torch.int32)
        if case["state"]:
            s["s0"] = rand(B, H, Dk, Dv, dtype=torch.float32)
        if op == "backward":
            s["do"] = rand(B, L, H, Dv)
            s["ds"] = rand(B, H, Dk, Dv, dtype=torch.float32) if case["state"] else None
        return s
    if op == "step":
        B, H, Hk, Dk, Dv = (case[n] for n in ("B", "H", "Hk", "Dk", "Dv"))
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        s = rand(B, H, Dk, Dv, dtype=torch.float32)
        return {"op": op, "q": rand(B, H, Dk, dtype=dt), "k": rand(B, Hk, Dk, dtype=dt),
                "v": rand(B, H, Dv, dtype=dt), "log_decay": _decay(H, g), "scale": Dk ** -0.5,
                "s": s, "s_next": torch.empty_like(s)}
    M, D = case["M"], case["D"]
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    s = {"op": op, "x": (torch.randn(M, D, device=DEV, generator=g) * 1.5 + 0.3).to(dt[case["x"]]),
         "w": 1 + 0.2 * torch.randn(D, device=DEV, generator=g),
         "b": 0.2 * torch.randn(D, device=DEV, generator=g), "eps": 1e-5, "y": dt[case["y"]]}
    if op == "norm_bwd":  # what the forward call leaves: the rows' mean and 1/std
        x = s["x"].double()
        s["mean"] = x.mean(-1).float()
        s["rstd"] = (x.var(-1, unbiased=False) + s["eps"]).rsqrt().float()
        s["dy"] = torch.randn(M, D, device=DEV, generator=g).to(s["y"])
    return s


# --------------------------------------------------------------------------- plain forms
def _pow(lam, n):
    """gamma^n from log gamma and exponents, in 64 bits (0^0 = 1)."""
    n = n.double()
    return torch.where(n == 0, torch.zeros_like(n), lam * n).exp()


def _heads(x, H):
    """[B, L, Hx, D] of any type -> [B, H, L, D] fp32, shared heads repeated."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2).contiguous()


def _causal(q, k, v, lam):
    """o_t = sum_{j <= t} gamma^(t-j) (q_t . k_j) v_j for [B, H, L, D] fp32, by chunks."""
    B, H, L, _ = q.shape
    C = min(128, L)
    N = -(-L // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, N * C - L)).unflatten(2, (N, C))
               for x in (q, k, v))
    i = torch.arange(C, device=q.device)
    lam = lam.double()[:, None, None]
    w = (_pow(lam, (i[:, None] - i).clamp_min(0)) * (i[:, None] >= i)).float()[:, None]
    o = ((q @ k.transpose(-1, -2)) * w) @ v
    if N > 1:
        kv = (k * _pow(lam, C - 1 - i[:, None]).float()[:, None]).transpose(-1, -2) @ v
        n = torch.arange(N, device=q.device)
        d = C * (n[:, None] - 1 - n)
        a = (_pow(lam, d.clamp_min(0)) * (d >= 0)).float()
        s = (a @ kv.flatten(3)).view_as(kv)
        o = o + (q * _pow(lam, i[:, None] + 1).float()[:, None]) @ s
    return o.flatten(2, 3)[:, :, :L]


def _live(s, L):
    """Lengths [B, 1, 1, 1] and the mask [B, 1, L, 1] of a batch's tokens."""
    B = s["q"].shape[0]
    t = torch.arange(L, device=s["q"].device)
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), L, device=t.device)
    n = n.view(B, 1, 1, 1)
    return n, t[:, None], t[:, None] < n


def _group(x, Hx):
    """Sum of [B, H, L, D] over the heads that share one -> [B, L, Hx, D] bf16."""
    return x.unflatten(1, (Hx, x.shape[1] // Hx)).sum(2).transpose(1, 2).bfloat16()


def _plain_scan(s):
    H, L = s["log_decay"].shape[0], s["q"].shape[1]
    n, t, live = _live(s, L)
    q, k, v = (_heads(s[x], H) * live for x in "qkv")
    lam = s["log_decay"].double()[:, None, None]
    o = _causal(q, k, v, s["log_decay"])
    fin = (k * _pow(lam, (n - 1 - t).clamp_min(0)).float()).transpose(-1, -2) @ v
    if s["s0"] is not None:
        o = o + (q * _pow(lam, t + 1).float()) @ s["s0"]
        fin = fin + _pow(lam, n).float() * s["s0"]
    return (o * s["scale"]).transpose(1, 2).bfloat16(), fin


def _plain_backward(s):
    H, L = s["log_decay"].shape[0], s["q"].shape[1]
    n, t, live = _live(s, L)
    q, k, v, do = (_heads(s[x], H) * live for x in ("q", "k", "v", "do"))
    lam = s["log_decay"].double()[:, None, None]
    do = do * s["scale"]
    dq = _causal(do, v, k, s["log_decay"])
    dk = _causal(v.flip(2), do.flip(2), q.flip(2), s["log_decay"]).flip(2)
    dv = _causal(k.flip(2), q.flip(2), do.flip(2), s["log_decay"]).flip(2)
    ds0 = (q * (_pow(lam, t + 1) * live).float()).transpose(-1, -2) @ do
    if s["s0"] is not None:
        dq = dq + (do * _pow(lam, t + 1).float()) @ s["s0"].transpose(-1, -2)
    if s["ds"] is not None:
        w = _pow(lam, (n - 1 - t).clamp_min(0)).float()
        dk = dk + (v * w) @ s["ds"].transpose(-1, -2)
        dv = dv + (k * w) @ s["ds"]
        ds0 = ds0 + _pow(lam, n).float() * s["ds"]
    return (_group(dq, s["q"].shape[2]), _group(dk, s["k"].shape[2]), _group(dv, s["v"].shape[2]),
            ds0)


def _plain_step(s):
    H = s["log_decay"].shape[0]
    q, k, v = (s[x].float().repeat_interleave(H // s[x].shape[1], dim=1) for x in "qkv")
    gamma = s["log_decay"].double().exp().float()[:, None, None]
    s_next = gamma * s["s"] + k[..., :, None] * v[..., None, :]
    o = (q[..., None, :] @ s_next).squeeze(-2) * s["scale"]
    s["s_next"].copy_(s_next)
    return o.to(s["q"].dtype), s["s_next"]


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = ((d * d).mean(-1, keepdim=True) + s["eps"]).rsqrt()
    return (d * rstd * s["w"] + s["b"]).to(s["y"]), mean.squeeze(-1), rstd.squeeze(-1)


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["w"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def run(state):
    op = state["op"]
    if own:
        import nonlinear_rnn_solve_newton_b200 as pr

        s = state
        if op == "scan":
            return pr.scan_linattn(s["q"], s["k"], s["v"], s["log_decay"], s["s0"],
                                   scale=s["scale"], lengths=s["lengths"])
        if op == "backward":
            return pr.scan_linattn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"],
                                            s0=s["s0"], ds=s["ds"], scale=s["scale"],
                                            lengths=s["lengths"])
        if op == "step":
            return pr.step_linattn(s["q"], s["k"], s["v"], s["log_decay"], s["s"],
                                   scale=s["scale"], state_out=s["s_next"])
        if op == "norm":
            return pr.layer_norm(s["x"], s["w"], s["b"], eps=s["eps"], out_dtype=s["y"])
        return pr.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    return {"scan": _plain_scan, "backward": _plain_backward, "step": _plain_step,
            "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[op](state)


# --------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("scan", "backward"):
        B, L, H, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "L", "H", "Hk", "Hv", "Dk", "Dv"))
        io = 2 * B * L * (H * Dk + Hk * Dk + Hv * Dv)
        st = 4 * B * H * Dk * Dv
        fl = 4 * B * L * H * Dk * Dv  # k^T v into the state, q times the state
        if op == "scan":
            return {"bytes": io + 2 * B * L * H * Dv + st * (2 if case["state"] else 1), "flops": fl}
        return {"bytes": 2 * io + 2 * B * L * H * Dv + st * (3 if case["state"] else 1),
                "flops": 3 * fl}
    if op == "step":
        B, H, Hk, Dk, Dv = (case[n] for n in ("B", "H", "Hk", "Dk", "Dv"))
        es = 4 if case["fp32"] else 2
        return {"bytes": 8 * B * H * Dk * Dv + es * B * (H * Dk + Hk * Dk + 2 * H * Dv),
                "flops": 5 * B * H * Dk * Dv}
    M, D = case["M"], case["D"]
    es = {"f32": 4, "bf16": 2}
    if op == "norm":
        return {"bytes": M * D * (es[case["x"]] + es[case["y"]]) + 8 * M + 8 * D, "flops": 8 * M * D}
    return {"bytes": M * D * (2 * es[case["x"]] + es[case["y"]]) + 8 * M + 12 * D,
            "flops": 14 * M * D}


# --------------------------------------------------------------------------- 64-bit definition
def _direct(q, k, v, lam, reverse):
    """sum over j <= t (reverse: j >= t) of gamma^|t-j| (q_t . k_j) v_j for one head, [L, D] in
    64 bits, straight from the definition, a block of rows at a time."""
    L = q.shape[0]
    o = torch.empty(L, v.shape[1], dtype=torch.float64, device=q.device)
    rows = max(1, min(L, (1 << 26) // L))
    j = torch.arange(L, device=q.device)
    for r in range(0, L, rows):
        t = j[r:r + rows, None]
        cols = slice(r, L) if reverse else slice(0, min(L, r + rows))
        dist = (j[cols] - t) if reverse else (t - j[cols])
        w = torch.where(dist > 0, lam * dist, torch.zeros((), dtype=torch.float64,
                                                          device=q.device)).exp()
        w = w.masked_fill_(dist < 0, 0.0)
        o[r:r + rows] = (w * (q[r:r + rows] @ k[cols].T)) @ v[cols]
    return o


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "backward"):
        B, L, H, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "L", "H", "Hk", "Hv", "Dk", "Dv"))
        f64 = dict(dtype=torch.float64, device=DEV)
        lens = [L] * B if s["lengths"] is None else s["lengths"].tolist()
        lam, c = s["log_decay"].double(), s["scale"]
        o, fin = torch.zeros(B, L, H, Dv, **f64), torch.zeros(B, H, Dk, Dv, **f64)
        dq, dk, dv = (torch.zeros(B, L, h, d, **f64) for h, d in ((H, Dk), (Hk, Dk), (Hv, Dv)))
        for b in range(B):
            n = lens[b]
            t = torch.arange(n, device=DEV, dtype=torch.float64)[:, None]
            for h in range(H):
                hk, hv = h * Hk // H, h * Hv // H
                q, k, v = (x.double() for x in (s["q"][b, :n, h], s["k"][b, :n, hk],
                                                s["v"][b, :n, hv]))
                before, after = (lam[h] * (t + 1)).exp(), (lam[h] * (n - 1 - t)).exp()
                if op == "scan":
                    y = _direct(q, k, v, lam[h], False)
                    fin[b, h] = (k * after).T @ v
                    if s["s0"] is not None:
                        s0 = s["s0"][b, h].double()
                        y += before * (q @ s0)
                        fin[b, h] += (lam[h] * n).exp() * s0
                    o[b, :n, h] = c * y
                    continue
                do = c * s["do"][b, :n, h].double()
                a, e, f = (_direct(do, v, k, lam[h], False), _direct(v, do, q, lam[h], True),
                           _direct(k, q, do, lam[h], True))
                fin[b, h] = (q * before).T @ do
                if s["s0"] is not None:
                    a += before * (do @ s["s0"][b, h].double().T)
                if s["ds"] is not None:
                    ds = s["ds"][b, h].double()
                    e += after * (v @ ds.T)
                    f += after * (k @ ds)
                    fin[b, h] += (lam[h] * n).exp() * ds
                dq[b, :n, h] += a
                dk[b, :n, hk] += e
                dv[b, :n, hv] += f
        return (o, fin) if op == "scan" else (dq, dk, dv, fin)
    if op == "step":
        H = case["H"]
        q, k, v = (s[x].double().repeat_interleave(H // s[x].shape[1], dim=1) for x in "qkv")
        nxt = s["s"].double() * s["log_decay"].double().exp()[:, None, None]
        nxt = nxt + torch.einsum("bhi,bhj->bhij", k, v)
        return torch.einsum("bhi,bhij->bhj", q, nxt) * s["scale"], nxt
    x = s["x"].double()
    if op == "norm":
        var, mean = torch.var_mean(x, -1, unbiased=False)
        rstd = 1 / torch.sqrt(var + s["eps"])
        y = torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double())
        return y, mean, rstd
    rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
    xh = (x - s["mean"].double()[:, None]) * rstd
    wdy = dy * s["w"].double()
    a = wdy.sum(-1, keepdim=True) / case["D"]
    b = (wdy * xh).sum(-1, keepdim=True) / case["D"]
    return (wdy - a - xh * b) * rstd, torch.einsum("md,md->d", dy, xh), dy.sum(0)
