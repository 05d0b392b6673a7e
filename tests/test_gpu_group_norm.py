"""Group norm with an activation, channels last, on the GPU against 64 bits (gradients by autograd in 64 bits)."""
import pytest
import torch

import layer_reference as ref
from xlstm_mlstm_matrix_b200 import capi

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def make(B, G, T, D, xd, yd, layout, gate, affine, seed=0, mean=0.3, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = (r(*((B, G, T, D) if layout == "heads" else (B, T, G, D))) * std + mean).to(xd)
    return dict(x=x, weight=1 + 0.2 * r(G * D) if affine else None, bias=0.1 * r(G * D) if affine else None,
                gate=(2 * r(B, T, G * D)).to(yd) if gate else None), r(B, T, G * D).to(yd)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def row_terms(s, layout, eps):
    """Per element of [B,T,G*D]: |xh|, and the error of xh: the mean is off by at most (D + 2) roundings of the largest
    magnitude of the row (a sum of D values), which shifts xh by that times rstd; centring, the variance (a sum of D
    squares: half its relative error), sqrt, division and product add D / 2 + 8 roundings of xh itself.  Sums run over
    32 lanes of at most 16 values, so 16 + 5 roundings stand in the place of D."""
    x = s["x"].double()
    x = x.transpose(1, 2) if layout == "heads" else x
    mu = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mu) * rstd
    shift = 24 * U * x.abs().amax(-1, keepdim=True) * rstd
    # a shifted mean changes the variance in second order only
    return xh.flatten(2), (shift + 24 * U * xh.abs()).flatten(2), rstd


def act_error(x):
    """Relative error of the sigmoid at x: the exponential's argument is rounded twice (|x| 2^-23), the base-2
    exponential and the division are good to 2^-22 each."""
    return x.abs() * 2.0 ** -23 + 2.0 ** -21 + 4 * U


def check(s, dy, act, layout, eps=1e-5):
    yd = dy.dtype
    y = capi.group_norm(**s, act=act, layout=layout, eps=eps, out_dtype=yd)
    g = capi.group_norm_bwd(dy, **s, act=act, layout=layout, eps=eps)
    leaves = {n: None if t is None else t.double().requires_grad_(True) for n, t in s.items()}
    want = ref.group_norm(leaves["x"], leaves["weight"], leaves["bias"], leaves["gate"], act, layout, eps)
    names = [n for n in leaves if leaves[n] is not None]
    grads = dict(zip(names, torch.autograd.grad(want, [leaves[n] for n in names], dy.double())))
    want = want.detach()
    xh, dxh, rstd = row_terms(s, layout, eps)
    w = torch.ones_like(xh) if s["weight"] is None else s["weight"].double().expand_as(xh)
    b = torch.zeros_like(xh) if s["bias"] is None else s["bias"].double().expand_as(xh)
    z, ez = xh * w + b, dxh * w.abs() + 2 * U * (xh * w).abs() + U * b.abs()
    pre = s["gate"].double() if s["gate"] is not None else z
    p = torch.sigmoid(pre)
    f = ref.act(pre, act)
    df = {"none": torch.ones_like(p), "sigmoid": p * (1 - p), "silu": p * (1 + pre * (1 - p))}[act]
    ef = torch.zeros_like(p) if act == "none" else f.abs() * act_error(pre)
    # act': p and 1 - p each off by p (1 - p) times the sigmoid's relative error and a rounding of 1
    edf = torch.zeros_like(p) if act == "none" else (act_error(pre) * p + 4 * U) * (2 + pre.abs())
    assert float(edf.max()) < 1e-3
    if s["gate"] is not None:
        ey = ez * f.abs() + z.abs() * ef + 2 * U * want.abs()
    else:
        ey = 1.2 * ez + ef + 2 * U * want.abs()          # |act'| <= 1.1
    near = lambda got, ref_, bound, what: _near(got, ref_, bound, what)  # noqa: E731
    near(y, want, ey + half_step(yd) * (want.abs() + ey), "y")
    d = dy.double()
    if s["gate"] is not None:
        dz, edz = d * f, d.abs() * ef + 2 * U * (d * f).abs()
        dgate = d * z * df
        eg = d.abs() * (ez * df.abs() + z.abs() * edf) + 3 * U * dgate.abs()
        near(g["dgate"], grads["gate"], eg + half_step(yd) * (dgate.abs() + eg), "dgate")
    else:
        dz = d * df
        # act'' <= 0.5 on these activations
        edz = d.abs() * (edf + 0.5 * ez) + 2 * U * dz.abs()
    n = d.shape[0] * d.shape[1]
    # sums over the tokens of terms each off by e: their errors and n roundings of the magnitudes' sum; in blocks of
    # at most sqrt-many, 600 roundings cover every order used here
    roundings = min(n, 600) + 16
    if s["weight"] is not None:
        t, e = dz * xh, edz * xh.abs() + dz.abs() * dxh
        near(g["dweight"], grads["weight"], e.sum((0, 1)) + roundings * U * t.abs().sum((0, 1)), "dweight")
        near(g["dbias"], grads["bias"], edz.sum((0, 1)) + roundings * U * dz.abs().sum((0, 1)), "dbias")
    G, D = rstd.shape[2], s["x"].shape[-1]
    view = lambda t: t.unflatten(2, (G, D))  # noqa: E731
    u, eu = view(dz * w), view(edz * w.abs() + U * (dz * w).abs())
    h, eh = view(xh), view(dxh)
    m1, m2 = u.mean(-1, keepdim=True), (u * h).mean(-1, keepdim=True)
    em1 = eu.mean(-1, keepdim=True) + 24 * U * u.abs().mean(-1, keepdim=True)
    em2 = (eu * h.abs() + u.abs() * eh).mean(-1, keepdim=True) + 24 * U * (u * h).abs().mean(-1, keepdim=True)
    inner = u - m1 - h * m2
    e = eu + em1 + h.abs() * em2 + eh * m2.abs() + 4 * U * (u.abs() + m1.abs() + (h * m2).abs())
    e = rstd * e + 32 * U * (rstd * inner).abs()
    dx = grads["x"].transpose(1, 2) if layout == "heads" else grads["x"]
    got = g["dx"].transpose(1, 2) if layout == "heads" else g["dx"]
    near(got, dx, e + half_step(s["x"].dtype) * (dx.abs() + e), "dx")
    return y, g


def _near(got, want, bound, what):
    d = (got.double() - want).abs()
    bad = ~(d <= bound + 1e-35)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / bound.clamp(min=1e-300)).max()):.3g} x bound"


DIMS = [16, 32, 48, 64, 80, 128, 144, 256, 272, 400, 512]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)], ids=["ff", "bb", "fb", "bf"])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gated"])
def test_group_norm(D, types, layout, gate):
    act = ("none", "silu", "sigmoid")[(D // 16 + gate) % 3]
    s, dy = make(2, 3, 41, D, *types, layout, gate, affine=(D // 16) % 4 != 0, seed=D)
    check(s, dy, act, layout)


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16), (1, 1, 1, 512), (3, 5, 1, 64), (1, 2, 1001, 96), (7, 1, 129, 32)], ids=str)
def test_sizes(act, gate, shape):
    s, dy = make(*shape, F32, F32, "heads", gate, True, seed=sum(shape))
    check(s, dy, act, "heads")


def test_large_mean_and_constant_rows():
    """A mean far above the spread; rows whose channels are all equal (variance 0: xh is 0, rstd is eps^-1/2)."""
    s, dy = make(2, 2, 33, 64, F32, F32, "tokens", True, True, seed=1, mean=1000.0, std=1.0)
    check(s, dy, "silu", "tokens")
    s, dy = make(2, 2, 33, 64, BF16, BF16, "tokens", True, True, seed=2)
    s["x"][0, 3] = 5.0
    s["x"][1, 7] = 0.0
    check(s, dy, "silu", "tokens")


def test_gate_extremes():
    """Gates at both ends: the activation saturates without NaN."""
    s, dy = make(1, 2, 4, 32, F32, F32, "heads", True, True, seed=3)
    s["gate"][0, 0] = 100.0
    s["gate"][0, 1] = -100.0
    s["gate"][0, 2] = 1e30
    s["gate"][0, 3] = -1e30
    for act in ("silu", "sigmoid"):
        y = capi.group_norm(**s, act=act)
        g = capi.group_norm_bwd(dy, **s, act=act)
        assert bool(torch.isfinite(y).all()) and all(bool(torch.isfinite(t).all()) for t in g.values())
        assert not y[0, 3].any()


def test_one_bad_row_stays_alone():
    """NaN in one token and head reaches that group's outputs and the sums over tokens, nothing else."""
    s, dy = make(2, 3, 40, 64, F32, F32, "heads", True, True, seed=4)
    y0, g0 = capi.group_norm(**s), capi.group_norm_bwd(dy, **s)
    s["x"][1, 2, 5, 7] = float("nan")
    y, g = capi.group_norm(**s), capi.group_norm_bwd(dy, **s)
    assert bool(torch.isnan(y[1, 5, 128:192]).all()) and bool(torch.isnan(g["dx"][1, 2, 5]).all())
    y[1, 5, 128:192] = y0[1, 5, 128:192]
    g["dx"][1, 2, 5] = g0["dx"][1, 2, 5]
    assert torch.equal(y, y0) and torch.equal(g["dx"], g0["dx"])
    assert torch.equal(g["dweight"][:128], g0["dweight"][:128])


def test_no_tokens():
    s, dy = make(2, 3, 0, 64, F32, F32, "heads", False, True)
    assert capi.group_norm(**s).shape == (2, 0, 192)
    g = capi.group_norm_bwd(dy, **s)
    assert not g["dweight"].any() and not g["dbias"].any()


def test_only_one_parameter():
    s, dy = make(2, 3, 50, 64, BF16, BF16, "heads", True, True, seed=6)
    full = capi.group_norm_bwd(dy, **dict(s, bias=torch.zeros_like(s["bias"])))
    g = capi.group_norm_bwd(dy, **dict(s, bias=None))
    assert g["dbias"] is None and torch.equal(g["dweight"], full["dweight"]) and torch.equal(g["dx"], full["dx"])
    g = capi.group_norm_bwd(dy, **dict(s, weight=None))
    assert g["dweight"] is None and g["dbias"].shape == (192,)


def test_streams_graph_repeatable():
    s, dy = make(4, 4, 700, 128, BF16, BF16, "heads", True, True, seed=8)
    y, g = capi.group_norm(**s), capi.group_norm_bwd(dy, **s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, g2 = capi.group_norm(**s, stream=side), capi.group_norm_bwd(dy, **s, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = capi.group_norm(**s), capi.group_norm_bwd(dy, **s)
    s["x"].mul_(0.5)
    dy.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    y, g = capi.group_norm(**s), capi.group_norm_bwd(dy, **s)
    assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)
