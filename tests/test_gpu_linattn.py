"""Linear attention with a decay per head on the GPU against the 64-bit recurrence, within derived rounding bounds
(layer_reference.output_bound, state_bound)."""
import pytest
import torch

import layer_reference as ref
from xlstm_mlstm_matrix_b200 import capi

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(B, H, T, dqk, dv, dtype, seed=0, state=True, lens=None, decay="mixed"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
    if decay == "mixed":      # memories from one token to thousands
        ld = -torch.exp2(-torch.linspace(-1.0, 12.0, H, device="cuda")) if H > 1 else torch.full((1,), -0.01, device="cuda")
    else:
        ld = torch.tensor([decay] * H, device="cuda", dtype=F32)
    x = dict(q=r(B, H, T, dqk), k=r(B, H, T, dqk), v=r(B, H, T, dv), log_decay=ld,
             state=r(B, H, dv, dqk, dt=F32) if state else None,
             lens=None if lens is None else torch.tensor(lens, device="cuda", dtype=torch.int32))
    x["do"] = r(B, H, T, dv)
    x["dstate"] = r(B, H, dv, dqk, dt=F32) if state else None
    return x


def status_ok(ws):
    code, where = capi.xlstm_mlstm_workspace_status(ws)
    assert code == capi.XLSTM_OK, (capi.xlstm_status_string(code), where)


def desc_of(x, scale):
    B, H, T, dqk = x["q"].shape
    return capi.make_linattn_desc(B, H, T, dqk, x["v"].shape[-1],
                                  capi.XLSTM_BF16 if x["q"].dtype == BF16 else capi.XLSTM_F32, scale)


def near(got, want, bound, what):
    """|got - want| <= bound, plus what fp32 loses below its range: a power of the decay under 2^-149 (or bf16 copy of
    one) becomes 0, off by at most 2^-133 (bf16's smallest step) before it meets values below 2^5 each in products of
    two and sums of up to 2^11 of them, 2^-133+10+11 < 2^-110 in all."""
    d = (got.double() - want).abs()
    bound = bound + 2.0 ** -110
    bad = ~(d <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / bound.clamp(min=1e-300)).max()):.3g} x bound"


def check_fwd(x, scale=None):
    dt, T, dqk = x["q"].dtype, x["q"].shape[2], x["q"].shape[3]
    scale = dqk ** -0.5 if scale is None else scale
    ws = torch.full((capi.xlstm_linattn_workspace_size(desc_of(x, scale)),), 0xFF, device="cuda", dtype=torch.uint8)
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    o, C = capi.linattn_fwd(*a, state=x["state"], lens=x["lens"], scale=scale, workspace=ws)
    status_ok(ws)
    want, mag = (f(*a, C0=x["state"], lens=x["lens"], scale=scale) for f in (ref.fwd, ref.fwd_magnitude))
    near(o, want[0], ref.output_bound(want[0], mag[0], T, dqk, dt), "o")
    near(C, want[1], ref.state_bound(mag[1], T, 0, dt), "C")
    return o, C


def check_bwd(x, scale=None):
    dt, T, dqk, dv = x["q"].dtype, x["q"].shape[2], x["q"].shape[3], x["v"].shape[3]
    scale = dqk ** -0.5 if scale is None else scale
    ws = torch.full((capi.xlstm_linattn_bwd_workspace_size(desc_of(x, scale)),), 0xFF, device="cuda", dtype=torch.uint8)
    a = (x["q"], x["k"], x["v"], x["log_decay"], x["do"])
    got = capi.linattn_bwd(*a, state=x["state"], dstate=x["dstate"], lens=x["lens"], scale=scale, workspace=ws)
    status_ok(ws)
    want, mag = (f(*a, C0=x["state"], dCT=x["dstate"], lens=x["lens"], scale=scale) for f in (ref.bwd, ref.bwd_magnitude))
    for n in ("dq", "dk", "dv"):
        near(got[n], want[n], ref.output_bound(want[n], mag[n], T, max(dqk, dv), dt), n)
    near(got["dC0"], want["dC0"], ref.state_bound(mag["dC0"], T, 0, dt), "dC0")
    return got


SHAPES = [  # B, H, T, dqk, dv
    (1, 1, 1, 16, 16), (2, 3, 2, 32, 48), (1, 2, 63, 64, 64), (1, 2, 64, 64, 64), (2, 1, 65, 64, 128), (1, 2, 127, 128, 64),
    (1, 2, 128, 128, 128), (1, 3, 129, 80, 96), (1, 2, 255, 256, 64), (1, 2, 257, 64, 256), (2, 2, 300, 112, 272),
    (1, 2, 511, 16, 512), (1, 1, 513, 512, 16), (1, 2, 640, 256, 512), (1, 1, 700, 512, 512), (3, 5, 1000, 64, 64),
    (1, 2, 1537, 128, 128),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_fwd(shape, dtype, state):
    check_fwd(make(*shape, dtype, seed=sum(shape), state=state))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_bwd(shape, dtype, state):
    check_bwd(make(*shape, dtype, seed=sum(shape) + 1, state=state))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(64, 64), (48, 80), (256, 128)], ids=str)
def test_padded_batch(dims, dtype):
    """Lengths of zero, one, around the tile and segment edges, out of range; NaN and infinities behind them."""
    T = 600
    lens = [0, 1, 63, 64, 65, 127, 128, 129, 200, 256, 257, 511, 512, 513, 599, 600, 601, -3]
    x = make(len(lens), 2, T, *dims, dtype, seed=9, lens=lens)
    for n, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", float("-inf"))):
        for b, m in enumerate(lens):
            x[n][b, :, max(0, min(m, T)):] = bad
    clean = dict(x)
    for n in ("q", "k", "v", "do"):
        clean[n] = torch.nan_to_num(x[n], 0.0, 0.0, 0.0)
    scale = dims[0] ** -0.5
    o, C = capi.linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"], lens=x["lens"], scale=scale)
    o2, C2 = check_fwd(clean, scale)
    assert torch.equal(o, o2) and torch.equal(C, C2)
    g = capi.linattn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["do"], state=x["state"], dstate=x["dstate"],
                         lens=x["lens"], scale=scale)
    g2 = check_bwd(clean, scale)
    for n in g:
        assert torch.equal(g[n], g2[n]), n
    for b, m in enumerate(lens):
        m = max(0, min(m, T))
        assert not o[b, :, m:].any() and not any(g[n][b, :, m:].any() for n in ("dq", "dk", "dv"))
    assert torch.equal(C[0], x["state"][0]) and torch.equal(g["dC0"][0], x["dstate"][0])


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
@pytest.mark.parametrize("shape", [(24, 3, 700, 64, 64), (9, 8, 600, 128, 96), (10, 6, 800, 256, 80), (7, 4, 780, 272, 160)], ids=str)
def test_many_heads(shape, state, ragged):
    """Heads enough for a block to carry a whole head's state, over more than two segments (bf16)."""
    lens = None
    if ragged:
        lens = ([shape[2], 0, 1, 255, 256, 257, 512, 513, 599] + list(range(300, 320)))[:shape[0]]
    x = make(*shape, BF16, seed=21, state=state, lens=lens)
    check_fwd(x)
    check_bwd(x)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 0.5, -1e-7, -0.69, -30.0, -1e30, float("-inf")])
def test_decays(decay, dtype):
    """No decay (and what is read as none), slow, fast, and no memory at all: finite and within the bound."""
    x = make(1, 2, 400, 64, 96, dtype, seed=4, decay=decay)
    check_fwd(x)
    check_bwd(x)


def test_scales():
    for scale in (0.0, -1.5):
        x = make(1, 2, 200, 64, 64, BF16, seed=5)
        check_fwd(x, scale)
        check_bwd(x, scale)


def test_no_tokens():
    for dtype in (F32, BF16):
        x = make(2, 2, 0, 64, 64, dtype)
        o, C = capi.linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state=x["state"])
        assert o.numel() == 0 and torch.equal(C, x["state"])
        g = capi.linattn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["do"], state=x["state"], dstate=x["dstate"])
        assert torch.equal(g["dC0"], x["dstate"])
        _, C = capi.linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"])
        assert not C.any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 16, 16), (2, 3, 48, 80), (1, 8, 128, 128), (3, 2, 256, 512), (2, 2, 512, 272),
                                   (40, 8, 64, 64), (1, 2, 400, 16)], ids=str)
@pytest.mark.parametrize("inplace", [False, True])
def test_step(shape, dtype, inplace):
    B, H, dqk, dv = shape
    x = make(B, H, 1, dqk, dv, dtype, seed=7)
    q, k, v = (x[n][:, :, 0].contiguous() for n in ("q", "k", "v"))
    C0 = x["state"].clone()
    o, C = capi.linattn_step(q, k, v, x["log_decay"], x["state"], inplace=inplace)
    assert (C.data_ptr() == x["state"].data_ptr()) == inplace
    assert inplace or torch.equal(x["state"], C0)
    scale = dqk ** -0.5
    a = (x["q"], x["k"], x["v"], x["log_decay"], C0, None, scale)
    want, mag = ref.fwd(*a), ref.fwd_magnitude(*a)
    u = dqk + 16
    b = u * 2.0 ** -24 * mag[0][:, :, 0]
    if dtype == BF16:
        b = b + 2.0 ** -8 * (want[0][:, :, 0].abs() + b)
    near(o, want[0][:, :, 0], b, "o")
    near(C, want[1], 16 * 2.0 ** -24 * mag[1], "C")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_prompt_then_tokens(dtype):
    """A prompt in one call, in two calls joined by the state, and a tail of single tokens agree with the recurrence."""
    x = make(2, 3, 330, 64, 128, dtype, seed=11)
    a = lambda s, e: tuple(x[n][:, :, s:e].contiguous() for n in ("q", "k", "v"))  # noqa: E731
    _, C = capi.linattn_fwd(*a(0, 200), x["log_decay"], state=x["state"])
    o2, C = capi.linattn_fwd(*a(200, 326), x["log_decay"], state=C)
    o = [o2]
    for t in range(326, 330):
        q, k, v = (y[:, :, 0].contiguous() for y in a(t, t + 1))
        o1, C = capi.linattn_step(q, k, v, x["log_decay"], C, inplace=True)
        o.append(o1[:, :, None])
    r = (x["q"], x["k"], x["v"], x["log_decay"], x["state"], None, 64 ** -0.5)
    want, mag = ref.fwd(*r), ref.fwd_magnitude(*r)
    near(torch.cat(o, 2), want[0][:, :, 200:], ref.output_bound(want[0], mag[0], 330, 64, dtype)[:, :, 200:], "o")
    near(C, want[1], 2 * ref.state_bound(mag[1], 330, 0, dtype), "C")


def test_optional_outputs():
    """Without a final state the outputs are the same bits; dC_in may be left out."""
    x = make(2, 2, 300, 64, 64, BF16, seed=13)
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    o, _ = capi.linattn_fwd(*a, state=x["state"])
    o2 = torch.empty_like(o)
    capi.linattn_fwd(*a, state=x["state"], out=(o2, None))
    assert torch.equal(o, o2)
    d = desc_of(x, 0.125)
    g = capi.linattn_bwd(*a, x["do"], state=x["state"], dstate=x["dstate"], scale=0.125)
    dq, dk, dv = torch.empty_like(x["q"]), torch.empty_like(x["k"]), torch.empty_like(x["v"])
    ws = torch.empty(capi.xlstm_linattn_bwd_workspace_size(d), device="cuda", dtype=torch.uint8)
    capi.check(capi.xlstm_linattn_bwd(d, *a, None, x["state"], x["do"], x["dstate"], dq, dk, dv, None, ws, ws.numel(),
                                      torch.cuda.current_stream()))
    assert all(torch.equal(p, g[n]) for p, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")))


def test_neighbours_untouched():
    """Nothing is written outside the outputs, the odd last rows included."""
    for dtype in (F32, BF16):
        x = make(1, 3, 201, 48, 80, dtype, seed=15)
        for n in (1, 2):
            buf = torch.full((x["v"].numel() + 512,), 7.0, device="cuda", dtype=dtype)
            o = buf[256:256 + x["v"].numel()].view_as(x["v"])
            cb = torch.full((3 * 80 * 48 + 512,), 7.0, device="cuda")
            C = cb[256:256 + 3 * 80 * 48].view(1, 3, 80, 48)
            capi.linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], out=(o, C))
            assert bool((buf[:256] == 7).all()) and bool((buf[-256:] == 7).all())
            assert bool((cb[:256] == 7).all()) and bool((cb[-256:] == 7).all())


def test_streams_and_graph():
    """The same bits on another stream, and replayed from a graph on changed inputs."""
    x = make(4, 2, 520, 128, 64, BF16, seed=17, lens=[520, 3, 0, 300])
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    kw = dict(state=x["state"], lens=x["lens"])
    o, C = capi.linattn_fwd(*a, **kw)
    g = capi.linattn_bwd(*a, x["do"], dstate=x["dstate"], **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, C2 = capi.linattn_fwd(*a, **kw, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(C, C2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gC = capi.linattn_fwd(*a, **kw)
        gg = capi.linattn_bwd(*a, x["do"], dstate=x["dstate"], **kw)
        so, sC = capi.linattn_step(*(y[:, :, 0].contiguous() for y in a[:3]), x["log_decay"], gC)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, go) and torch.equal(C, gC) and all(torch.equal(g[n], gg[n]) for n in g)
    for n in ("q", "k", "v", "do"):
        x[n].mul_(-0.5)
    x["lens"].copy_(torch.tensor([5, 520, 256, 0]))
    graph.replay()
    torch.cuda.synchronize()
    o, C = capi.linattn_fwd(*a, **kw)
    g = capi.linattn_bwd(*a, x["do"], dstate=x["dstate"], **kw)
    assert torch.equal(o, go) and torch.equal(C, gC) and all(torch.equal(g[n], gg[n]) for n in g)
    s2, _ = capi.linattn_step(*(y[:, :, 0].contiguous() for y in a[:3]), x["log_decay"], gC)
    assert torch.equal(so, s2)


def test_repeatable():
    x = make(2, 4, 1100, 128, 256, BF16, seed=19)
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    o, C = capi.linattn_fwd(*a, state=x["state"])
    g = capi.linattn_bwd(*a, x["do"], state=x["state"], dstate=x["dstate"])
    for _ in range(20):
        o2, C2 = capi.linattn_fwd(*a, state=x["state"])
        g2 = capi.linattn_bwd(*a, x["do"], state=x["state"], dstate=x["dstate"])
        assert torch.equal(o, o2) and torch.equal(C, C2) and all(torch.equal(g[n], g2[n]) for n in g)
