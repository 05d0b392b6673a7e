"""What is measured of the linear attention with a decay per head and of the group norm with an activation.

Linear attention: C_t = l C_{t-1} + v_t k_t^T, o_t = scale C_t q_t with l = exp(log_decay[h]) <= 1, as a whole prompt
(``linattn_fwd``), as one token per sequence (``linattn_step``) and its gradients (``linattn_bwd``).  Group norm: each
head's channels of a token are normalised, scaled and shifted, then multiplied by an activated gate (or activated) and
stored channels last (``group_norm``), and its gradients (``group_norm_bwd``).

With ``own`` false the operators run in their plain form (elementary torch operations in fp32); with ``own`` true
through the library's calls.
"""
import math

import torch

own = False

L = 64   # tokens of one chunk of the plain form


def listed():
    return [
        # prompt of a 7B-like layer, a batch of 4096-token prompts; the state goes on to the decode calls
        dict(name="fwd_layer_7b", op="linattn_fwd", B=8, H=8, T=4096, dqk=256, dv=512, dtype="bf16", state=False, lens=False),
        # one long document continued from a state, few heads
        dict(name="fwd_long_context", op="linattn_fwd", B=1, H=8, T=65536, dqk=128, dv=128, dtype="bf16", state=True, lens=False),
        # many short prompts of different lengths in one padded batch, small heads
        dict(name="fwd_many_short_ragged", op="linattn_fwd", B=256, H=4, T=512, dqk=64, dv=64, dtype="bf16", state=False, lens=True),
        # a tiny fp32 layer: the latency of a call
        dict(name="fwd_tiny_fp32", op="linattn_fwd", B=1, H=2, T=256, dqk=64, dv=64, dtype="fp32", state=False, lens=False),
        # decode of a served batch of the 7B-like layer
        dict(name="step_decode", op="linattn_step", B=128, H=8, dqk=256, dv=512, dtype="bf16"),
        # decode of one user's sequence: the latency of a call
        dict(name="step_one_user", op="linattn_step", B=1, H=8, dqk=128, dv=128, dtype="bf16"),
        # training step of the 7B-like layer
        dict(name="bwd_layer_7b", op="linattn_bwd", B=8, H=8, T=4096, dqk=256, dv=512, dtype="bf16", state=False, lens=False),
        # fp32 training of a small layer: odd length, head sizes that are not powers of two, continued from a state
        dict(name="bwd_odd_fp32", op="linattn_bwd", B=2, H=3, T=777, dqk=80, dv=96, dtype="fp32", state=True, lens=True),
        # the 7B-like layer's norm and SiLU gate after the cell's heads-major output
        dict(name="norm_layer_7b", op="group_norm", B=8, H=8, T=4096, D=512, x="bf16", y="bf16", layout="heads", gate=True, act="silu", affine=True),
        # the same stage of one decode step of a served batch, on the cell's fp32 output
        dict(name="norm_decode", op="group_norm", B=128, H=8, T=1, D=512, x="fp32", y="bf16", layout="heads", gate=True, act="sigmoid", affine=True),
        # its gradients in the training step
        dict(name="norm_bwd_layer_7b", op="group_norm_bwd", B=8, H=8, T=4096, D=512, x="bf16", y="bf16", layout="heads", gate=True, act="silu", affine=True),
        # fp32 training of a small layer, channels-last input, activation on the norm itself
        dict(name="norm_bwd_odd_fp32", op="group_norm_bwd", B=3, H=5, T=1001, D=80, x="fp32", y="fp32", layout="tokens", gate=False, act="silu", affine=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(2 ** rng.uniform(math.log2(lo), math.log2(hi))))))


def _too_much(c):
    heads, n = c["B"] * c["H"], -(-c["T"] // L)
    size, area = c["dqk"] + c["dv"], c["dqk"] * c["dv"]
    scale = 8 if c["dtype"] == "fp32" else 1
    return (scale * heads * c["T"] * size > 8 * 8 * 4096 * 768 or scale * heads * n * area > 8 * 8 * 64 * 256 * 512
            or heads * n * n * area > 8 * 1024 * 1024 * 128 * 128)


def draw(rng):
    op = rng.choice(["linattn_fwd", "linattn_fwd", "linattn_step", "linattn_bwd", "group_norm", "group_norm_bwd"])
    H = rng.randint(1, 16)
    if op.startswith("linattn"):
        c = dict(op=op, B=_log_int(rng, 1, 64), H=H, T=_log_int(rng, 1, 65536), dqk=16 * _log_int(rng, 1, 32),
                 dv=16 * _log_int(rng, 1, 32), dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]))
        if op == "linattn_step":
            del c["T"]
            c["B"] = _log_int(rng, 1, 256)
            while c["B"] * c["H"] * c["dqk"] * c["dv"] > 128 * 8 * 256 * 512:
                c["B"] = max(1, c["B"] * 3 // 4)
            return c
        while _too_much(c):
            if c["B"] > 1 and rng.random() < 0.5:
                c["B"] = c["B"] * 3 // 4
            else:
                c["T"] = max(1, c["T"] * 3 // 4)
        return dict(c, state=rng.random() < 0.5, lens=rng.random() < 0.4)
    c = dict(op=op, B=_log_int(rng, 1, 128), H=H, T=_log_int(rng, 1, 8192), D=16 * _log_int(rng, 1, 32),
             x=rng.choice(["bf16", "fp32"]), y=rng.choice(["bf16", "fp32"]), layout=rng.choice(["heads", "tokens"]),
             gate=rng.random() < 0.7, act=rng.choice(["none", "silu", "sigmoid"]), affine=rng.random() < 0.7)
    while c["B"] * c["H"] * c["T"] * c["D"] > 8 * 8 * 4096 * 512 // 2:
        c["T"], c["B"] = max(1, c["T"] * 3 // 4), max(1, c["B"] * 7 // 8)
    return c


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype="fp32", std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(_dtype(dtype))

    c = case
    B, H = c["B"], c["H"]
    s = dict(case)
    if c["op"].startswith("linattn"):
        dqk, dv, dt = c["dqk"], c["dv"], c["dtype"]
        # retention-like decays: memories of a few tokens in the first heads, of thousands in the last ones
        u = torch.linspace(1.0, 12.0, H, device="cuda") if H > 1 else torch.full((1,), 7.0, device="cuda")
        s["log_decay"] = -torch.exp2(-u - torch.rand(H, device="cuda", generator=gen))
        s["scale"] = dqk ** -0.5
        T = () if c["op"] == "linattn_step" else (c["T"],)
        s["q"], s["k"] = normal(B, H, *T, dqk, dtype=dt), normal(B, H, *T, dqk, dtype=dt)
        s["v"] = normal(B, H, *T, dv, dtype=dt)
        if c["op"] == "linattn_step":
            s["C"] = normal(B, H, dv, dqk)
            return s
        s["C"] = normal(B, H, dv, dqk) if c["state"] else None
        if c["lens"]:   # one sequence fills the batch, the others end anywhere, before their first token too
            s["lens"] = torch.randint(0, c["T"] + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
            s["lens"][0] = c["T"]
        else:
            s["lens"] = None
        if c["op"] == "linattn_bwd":
            s["do"] = normal(B, H, *T, dv, dtype=dt)
            s["dC"] = normal(B, H, dv, dqk) if c["state"] else None
        return s
    T, D = c["T"], c["D"]
    shape = (B, H, T, D) if c["layout"] == "heads" else (B, T, H, D)
    s["x"] = (torch.randn(*shape, device="cuda", generator=gen) * 2.0 + 0.3).to(_dtype(c["x"]))
    s["weight"] = 1.0 + 0.2 * normal(H * D) if c["affine"] else None
    s["bias"] = 0.1 * normal(H * D) if c["affine"] else None
    s["g"] = normal(B, T, H * D, dtype=c["y"]) if c["gate"] else None
    if c["op"] == "group_norm_bwd":
        s["dy"] = normal(B, T, H * D, dtype=c["y"])
    return s


# ---- plain forms: elementary torch operations in fp32 ---------------------------------------------------------
def _power(log_decay, n):
    """exp(log_decay n) for whole distances n >= 0, formed in 64 bits: [H, *n.shape] fp32."""
    ld = log_decay.double().reshape(-1, *([1] * n.dim()))
    return torch.exp(ld * n.double()).float()


def _chunks(x, n):
    """[B,H,T,d] -> [B,H,n,L,d] in fp32, zeros behind the end."""
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, n * L - x.shape[2]))
    return x.reshape(x.shape[0], x.shape[1], n, L, x.shape[3])


def _masked(x, lens):
    if lens is None:
        return x
    live = torch.arange(x.shape[2], device=x.device) < lens[:, None]
    return torch.where(live[:, None, :, None], x, torch.zeros((), device=x.device, dtype=x.dtype))


def _left(s):
    """Distance of each token to the last one of its sequence [B,T], and the sequences' lengths [B]."""
    T = s["q"].shape[2]
    lens = torch.full((s["q"].shape[0],), T, device=s["q"].device) if s["lens"] is None else s["lens"].long()
    return (lens[:, None] - 1 - torch.arange(T, device=s["q"].device)).clamp(min=0), lens


def _weights_to_end(s):
    left, lens = _left(s)
    return _power(s["log_decay"], left).transpose(0, 1), _power(s["log_decay"], lens).transpose(0, 1)   # [B,H,T], [B,H]


def _carry(ld, n):
    """Weights [H, n, n] of chunk m's sum in the state that chunk c starts from: l^(L (c-1-m)) for m < c."""
    c, m = torch.arange(n, device=ld.device)[:, None], torch.arange(n, device=ld.device)[None]
    return _power(ld, (L * (c - 1 - m)).clamp(min=0)) * (m < c)


def _plain_parts(s):
    q, k, v = (_masked(s[x], s["lens"]) for x in ("q", "k", "v"))
    ld, n = s["log_decay"], -(-q.shape[2] // L)
    i = torch.arange(L, device=q.device)
    mask = _power(ld, (i[:, None] - i[None]).clamp(min=0)) * (i[:, None] >= i[None])
    qc, kc, vc = _chunks(q, n), _chunks(k, n), _chunks(v, n)
    into = _power(ld, i + 1)[:, None, :, None]         # decay of the entering state at token i
    out = _power(ld, L - 1 - i)[:, None, :, None]      # decay of token i at the chunk's end
    U = (vc * out).transpose(-1, -2) @ kc              # [B,H,n,dv,dqk]
    states = (_carry(ld, n) @ U.flatten(3)).unflatten(3, U.shape[3:])
    if s["C"] is not None:
        states = states + _power(ld, L * torch.arange(n, device=q.device))[:, :, None, None] * s["C"][:, :, None]
    return qc, kc, vc, mask[:, None], into, out, states


def _unchunk(x, s, like):
    B, H, T = s["q"].shape[:3]
    return _masked(x.reshape(B, H, -1, x.shape[-1])[:, :, :T], s["lens"]).to(like.dtype)


def _plain_fwd(s):
    qc, kc, vc, mask, into, _, states = _plain_parts(s)
    o = ((qc @ kc.transpose(-1, -2)) * mask) @ vc + into * (qc @ states.transpose(-1, -2))
    w, whole = _weights_to_end(s)
    C = (_masked(s["v"], s["lens"]).float() * w[..., None]).transpose(-1, -2) @ _masked(s["k"], s["lens"]).float()
    if s["C"] is not None:
        C = C + whole[..., None, None] * s["C"]
    return _unchunk(s["scale"] * o, s, s["q"]), C


def _plain_step(s):
    k, v, q = s["k"].float(), s["v"].float(), s["q"].float()
    C = s["C"]
    C.mul_(torch.exp(s["log_decay"])[:, None, None]).addcmul_(v[..., :, None], k[..., None, :])
    return (s["scale"] * (C @ q[..., None])[..., 0]).to(s["q"].dtype), C


def _plain_bwd(s):
    qc, kc, vc, mask, into, out, states = _plain_parts(s)
    ld, a, n = s["log_decay"], s["scale"], qc.shape[2]
    do = _masked(s["do"], s["lens"])
    dc = _chunks(do, n)
    dS = (dc @ vc.transpose(-1, -2)) * mask
    S = (qc @ kc.transpose(-1, -2)) * mask
    G = a * (dc * into).transpose(-1, -2) @ qc          # this chunk's part of the adjoint at its start
    back = _carry(ld, n).transpose(-1, -2)              # from the chunks behind
    E = (back @ G.flatten(3)).unflatten(3, G.shape[3:])
    dq = a * (dS @ kc + into * (dc @ states))
    dk = a * (dS.transpose(-1, -2) @ qc) + out * (vc @ E)
    dv = a * (S.transpose(-1, -2) @ dc) + out * (kc @ E.transpose(-1, -2))
    ends = torch.arange(1, s["q"].shape[2] + 1, device=ld.device)
    dC = a * (do.float() * _power(ld, ends)[..., None]).transpose(-1, -2) @ _masked(s["q"], s["lens"]).float()
    dk, dv = (x.reshape(*x.shape[:2], -1, x.shape[-1])[:, :, :s["q"].shape[2]] for x in (dk, dv))
    if s["dC"] is not None:
        w, whole = _weights_to_end(s)
        dk = dk + w[..., None] * (_masked(s["v"], s["lens"]).float() @ s["dC"])
        dv = dv + w[..., None] * (_masked(s["k"], s["lens"]).float() @ s["dC"].transpose(-1, -2))
        dC = dC + whole[..., None, None] * s["dC"]
    return dict(dq=_unchunk(dq, s, s["q"]), dk=_unchunk(dk, s, s["k"]), dv=_unchunk(dv, s, s["v"]), dC0=dC)


EPS = 1e-5


def _act(x, act):
    return x if act == "none" else torch.sigmoid(x) if act == "sigmoid" else x * torch.sigmoid(x)


def _act_slope(x, act):
    p = torch.sigmoid(x)
    return torch.ones_like(x) if act == "none" else p * (1 - p) if act == "sigmoid" else p * (1 + x * (1 - p))


def _plain_normed(s):
    x = s["x"].float()
    x = x.transpose(1, 2) if s["layout"] == "heads" else x      # [B,T,H,D]
    centred = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(centred.square().mean(-1, keepdim=True) + EPS)
    return centred * rstd, rstd


def _plain_norm(s):
    xh, _ = _plain_normed(s)
    z = xh.flatten(2)
    if s["weight"] is not None:
        z = z * s["weight"] + s["bias"]
    y = _act(z, s["act"]) if s["g"] is None else z * _act(s["g"].float(), s["act"])
    return y.to(_dtype(s["y"]))


def _plain_norm_bwd(s):
    xh, rstd = _plain_normed(s)
    dy = s["dy"].float()
    z = xh.flatten(2)
    if s["weight"] is not None:
        z = z * s["weight"] + s["bias"]
    if s["g"] is None:
        dz, dgate = dy * _act_slope(z, s["act"]), None
    else:
        g = s["g"].float()
        dz, dgate = dy * _act(g, s["act"]), (dy * z * _act_slope(g, s["act"])).to(s["g"].dtype)
    dw = (dz * xh.flatten(2)).sum((0, 1)) if s["weight"] is not None else None
    db = dz.sum((0, 1)) if s["weight"] is not None else None
    dxh = (dz if s["weight"] is None else dz * s["weight"]).unflatten(2, xh.shape[2:])
    dx = rstd * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True))
    dx = dx.transpose(1, 2).contiguous() if s["layout"] == "heads" else dx
    return dict(dx=dx.to(s["x"].dtype), dgate=dgate, dweight=dw, dbias=db)


def run(state):
    s, op = state, state["op"]
    if own:
        from xlstm_mlstm_matrix_b200 import capi
        if op == "linattn_fwd":
            return capi.linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], state=s["C"], lens=s["lens"], scale=s["scale"])
        if op == "linattn_step":
            return capi.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["C"], scale=s["scale"], inplace=True)
        if op == "linattn_bwd":
            return capi.linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], state=s["C"], dstate=s["dC"],
                                    lens=s["lens"], scale=s["scale"])
        if op == "group_norm":
            return capi.group_norm(s["x"], s["weight"], s["bias"], gate=s["g"], act=s["act"], layout=s["layout"], eps=EPS,
                                   out_dtype=_dtype(s["y"]))
        return capi.group_norm_bwd(s["dy"], s["x"], s["weight"], s["bias"], gate=s["g"], act=s["act"],
                                   layout=s["layout"], eps=EPS)
    return {"linattn_fwd": _plain_fwd, "linattn_step": _plain_step, "linattn_bwd": _plain_bwd,
            "group_norm": _plain_norm, "group_norm_bwd": _plain_norm_bwd}[op](s)


def work(case):
    c = case
    if c["op"].startswith("linattn"):
        dqk, dv, heads = c["dqk"], c["dv"], c["B"] * c["H"]
        e, area = 2 if c["dtype"] == "bf16" else 4, 4 * c["dqk"] * c["dv"]
        if c["op"] == "linattn_step":
            return dict(bytes=heads * (e * (2 * dqk + 2 * dv) + 2 * area), flops=heads * 5 * dqk * dv)
        T = c["T"]
        # a padded batch is half filled on average
        tokens = heads * ((T + (c["B"] - 1) * T / 2) / c["B"] if c["lens"] else T)
        pairs = min(T, L)
        if c["op"] == "linattn_fwd":
            return dict(bytes=tokens * e * (2 * dqk + dv) + heads * T * e * dv + heads * area * (1 + c["state"]),
                        flops=tokens * (4 * dqk * dv + pairs * (dqk + dv)))
        return dict(bytes=tokens * e * (2 * dqk + 2 * dv) + heads * T * e * (2 * dqk + dv) + heads * area * (1 + 2 * c["state"]),
                    flops=tokens * (10 * dqk * dv + pairs * (3 * dqk + 2 * dv)))
    n = c["B"] * c["T"] * c["H"] * c["D"]
    ex, ey = (2 if c[x] == "bf16" else 4 for x in ("x", "y"))
    par = c["H"] * c["D"] * 8 * c["affine"]
    if c["op"] == "group_norm":
        return dict(bytes=n * (ex + ey * (1 + c["gate"])) + par, flops=12 * n)
    return dict(bytes=n * (2 * ex + ey * (1 + 2 * c["gate"])) + 2 * par, flops=24 * n)


# ---- the definitions in 64 bits -------------------------------------------------------------------------------
def _recurrence(s, q, k, v, C):
    """o and the last state, 128 tokens at a time, from the recurrence's unrolled form."""
    B, H, T, dqk = q.shape
    ld = s["log_decay"].double()[None, :, None]
    ends = torch.full((B,), T, device=q.device) if s["lens"] is None else s["lens"].long()
    pos = torch.arange(T, device=q.device)
    live = (pos < ends[:, None])[:, None, :, None]
    zero = torch.zeros((), device=q.device, dtype=torch.float64)
    q, k, v = (torch.where(live, x, zero) for x in (q, k, v))
    C = torch.zeros(B, H, v.shape[-1], dqk, device=q.device, dtype=torch.float64) if C is None else C
    o = []
    for t0 in range(0, T, 128):
        qb, kb, vb = (x[:, :, t0:t0 + 128] for x in (q, k, v))
        i = torch.arange(qb.shape[2], device=q.device)
        far = (i[:, None] - i[None]).double()
        w = torch.where(far >= 0, torch.exp(ld[..., None] * far.clamp(min=0)), zero)
        o.append(torch.einsum("bhts,bhsv->bhtv", torch.einsum("bhtd,bhsd->bhts", qb, kb) * w, vb)
                 + torch.exp(ld * (i + 1).double())[..., None] * torch.einsum("bhtd,bhvd->bhtv", qb, C))
        here = (ends - t0).clamp(0, qb.shape[2]).double()[:, None, None]            # live tokens of this block
        rest = (here - 1 - i.double()).clamp(min=0)
        C = torch.exp(ld * here)[..., None] * C + torch.einsum("bhsv,bhsd->bhvd", vb * torch.exp(ld * rest)[..., None], kb)
    return torch.where(live, s["scale"] * torch.cat(o, 2), zero), C


def _exact_norm(s, x, w, b, g):
    xt = x.permute(0, 2, 1, 3) if s["layout"] == "heads" else x
    mu = xt.mean(-1, keepdim=True)
    var = (xt * xt).mean(-1, keepdim=True) - mu * mu
    z = ((xt - mu) / torch.sqrt(var + EPS)).reshape(*xt.shape[:2], -1)
    if w is not None:
        z = z * w + b
    f = {"none": lambda t: t, "sigmoid": lambda t: 1 / (1 + torch.exp(-t)), "silu": lambda t: t / (1 + torch.exp(-t))}[s["act"]]
    return f(z) if g is None else z * f(g)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = lambda x, grad=False: None if s.get(x) is None else s[x].double().requires_grad_(grad)  # noqa: E731
    if op == "linattn_fwd":
        return _recurrence(s, d("q"), d("k"), d("v"), d("C"))
    if op == "linattn_step":
        C = torch.exp(s["log_decay"].double())[:, None, None] * d("C") + d("v")[..., :, None] * d("k")[..., None, :]
        return s["scale"] * torch.einsum("bhvd,bhd->bhv", C, d("q")), C
    if op == "linattn_bwd":
        B, H, _, dqk = s["q"].shape
        C0 = s["C"].double() if s["C"] is not None else torch.zeros(B, H, s["v"].shape[-1], dqk, device="cuda", dtype=torch.float64)
        ins = [d("q", True), d("k", True), d("v", True), C0.requires_grad_(True)]
        o, C = _recurrence(s, *ins)
        up = torch.zeros_like(C) if s["dC"] is None else s["dC"].double()
        return dict(zip(("dq", "dk", "dv", "dC0"), torch.autograd.grad([o, C], ins, [d("do"), up])))
    if op == "group_norm":
        return _exact_norm(s, d("x"), d("weight"), d("bias"), d("g"))
    ins = [d("x", True), d("weight", True), d("bias", True), d("g", True)]
    y = _exact_norm(s, *ins)
    got = iter(torch.autograd.grad(y, [x for x in ins if x is not None], d("dy")))
    gx, gw, gb, gg = (None if x is None else next(got) for x in ins)
    return dict(dx=gx, dgate=gg, dweight=gw, dbias=gb)
