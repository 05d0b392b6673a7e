"""The layer operators as they are used together, and at the ends of their ranges.

Chains are checked stage by stage: every operator against 64 bits on the very inputs that the one before it wrote, within
its own rounding bounds.  Large calls are checked against small ones on a part of their data."""
import pytest
import torch

import layer_reference as ref
from test_gpu_group_norm import check as check_norm
from test_gpu_linattn import check_bwd, check_fwd, make, near
from xlstm_mlstm_matrix_b200 import capi

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def normal(*shape, dtype=F32, seed=0):
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


def affine(C):
    return dict(weight=1 + 0.2 * normal(C, seed=101), bias=0.1 * normal(C, seed=102))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(2, 3, 333, 64, 96), (1, 4, 520, 128, 256)], ids=str)
def test_training_step(dims, dtype):
    """Attention, norm and gate forwards, then their gradients backwards."""
    B, H, T, dqk, dv = dims
    x = make(*dims, dtype, seed=3)
    o, _ = check_fwd(x)
    s = dict(x=o, **affine(H * dv), gate=normal(B, T, H * dv, dtype=dtype, seed=4))
    _, g = check_norm(s, normal(B, T, H * dv, dtype=dtype, seed=5), "silu", "heads")
    assert g["dx"].shape == o.shape and g["dx"].dtype == o.dtype
    x["do"] = g["dx"]
    check_bwd(x)


def test_training_step_captured():
    """The whole step in one graph, replayed on changed inputs, gives an eager step's bits."""
    B, H, T, dqk, dv = 2, 4, 600, 64, 128
    x = make(B, H, T, dqk, dv, BF16, seed=6, lens=[600, 77])
    a, kw = (x["q"], x["k"], x["v"], x["log_decay"]), dict(state=x["state"], lens=x["lens"])
    w, gate, dy = affine(H * dv), normal(B, T, H * dv, dtype=BF16, seed=7), normal(B, T, H * dv, dtype=BF16, seed=8)

    def step():
        o, C = capi.linattn_fwd(*a, **kw)
        y = capi.group_norm(o, **w, gate=gate)
        g = capi.group_norm_bwd(dy, o, **w, gate=gate)
        return [y, C, *g.values(), *capi.linattn_bwd(*a, g["dx"], dstate=x["dstate"], **kw).values()]

    eager = step()      # its tensors stay alive while the graph is captured
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for change in range(2):
        if change:
            for t in (x["q"], x["v"], gate, dy):
                t.mul_(-0.75)
            x["lens"].copy_(torch.tensor([0, 600]))
            eager = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(eager, captured))


def test_decode():
    """A prompt, then single tokens in place, each through the norm: the same rows as the whole sequence gives."""
    B, H, T, dqk, dv = 3, 2, 150, 64, 64
    x = make(B, H, T, dqk, dv, F32, seed=9, state=False)
    w = affine(H * dv)
    a = (x["q"], x["k"], x["v"])
    _, C = capi.linattn_fwd(*(t[:, :, :140].contiguous() for t in a), x["log_decay"])
    want, mag = (f(*a, x["log_decay"], scale=dqk ** -0.5) for f in (ref.fwd, ref.fwd_magnitude))
    for t in range(140, T):
        o, C = capi.linattn_step(*(t_[:, :, t].contiguous() for t_ in a), x["log_decay"], C, inplace=True)
        near(o, want[0][:, :, t], ref.output_bound(want[0], mag[0], T, dqk, F32)[:, :, t], "o")
        check_norm(dict(x=o.view(B, H, 1, dv), **w, gate=normal(B, 1, H * dv, dtype=BF16, seed=t)),
                   normal(B, 1, H * dv, dtype=BF16, seed=t + 1), "sigmoid", "heads")


def test_cell_then_norm():
    """The mLSTM cell's fp32 output through the norm into bf16, and the gradient back into the cell."""
    B, H, T, dqk, dv = 2, 4, 256, 64, 128
    q, k, v = (normal(B, H, T, d, dtype=BF16, seed=10 + i) for i, d in enumerate((dqk, dqk, dv)))
    i_pre, f_pre = normal(B, H, T, seed=13), normal(B, H, T, seed=14) + 3
    h, _ = capi.fwd(q, k, v, i_pre, f_pre)
    s = dict(x=h, **affine(H * dv), gate=normal(B, T, H * dv, dtype=BF16, seed=15))
    _, g = check_norm(s, normal(B, T, H * dv, dtype=BF16, seed=16), "sigmoid", "heads")
    grads = capi.bwd(q, k, v, i_pre, f_pre, g["dx"])
    assert all(bool(torch.isfinite(t).all()) for t in grads.values())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_two_calls_at_once(dtype):
    """Calls on two streams, a workspace each, do not touch one another."""
    xs = [make(4, 4, 700, 128, 128, dtype, seed=20 + i) for i in range(2)]
    norms = [dict(x=normal(4, 4, 700, 128, dtype=dtype, seed=30 + i), **affine(512)) for i in range(2)]
    dys = [normal(4, 700, 512, dtype=dtype, seed=40 + i) for i in range(2)]

    def calls(i, **kw):
        x = xs[i]
        a = (x["q"], x["k"], x["v"], x["log_decay"])
        return [*capi.linattn_fwd(*a, state=x["state"], **kw),
                *capi.linattn_bwd(*a, x["do"], state=x["state"], dstate=x["dstate"], **kw).values(),
                *(t for t in capi.group_norm_bwd(dys[i], **norms[i], **kw).values() if t is not None)]

    want = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(5):
        got = [calls(i, stream=streams[i] if k % 2 else streams[i].cuda_stream) for i in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for i in range(2) for p, q in zip(want[i], got[i]))


def test_memory_of_another_stream():
    """A helper's workspace stays the call's own until the other stream is done, whatever is allocated meanwhile."""
    x = make(2, 4, 2000, 64, 64, BF16, seed=50, state=False)
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    want = capi.linattn_fwd(*a)
    g = capi.linattn_bwd(*a, x["do"])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)      # some 25 ms
    o, C = capi.linattn_fwd(*a, stream=side)
    g2 = capi.linattn_bwd(*a, x["do"], stream=side)
    d = capi.make_linattn_desc(2, 4, 2000, 64, 64, capi.XLSTM_BF16, 0.125)
    for n in (capi.xlstm_linattn_workspace_size(d), capi.xlstm_linattn_bwd_workspace_size(d)):
        for _ in range(3):
            torch.empty(n, device="cuda", dtype=torch.uint8).fill_(0x7F)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(C, want[1]) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_no_sequence_has_a_token(dtype):
    x = make(3, 2, 200, 64, 64, dtype, seed=60, lens=[0, -5, 0])
    for n in ("q", "k", "v", "do"):
        x[n].fill_(float("nan"))
    a, kw = (x["q"], x["k"], x["v"], x["log_decay"]), dict(state=x["state"], lens=x["lens"])
    o, C = capi.linattn_fwd(*a, **kw)
    g = capi.linattn_bwd(*a, x["do"], dstate=x["dstate"], **kw)
    assert not bool(o.any()) and torch.equal(C, x["state"])
    assert not any(bool(g[n].any()) for n in ("dq", "dk", "dv")) and torch.equal(g["dC0"], x["dstate"])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_views(dtype):
    """Decays and lengths at any 4-byte address, the other tensors at any 16-byte address."""
    x = make(3, 2, 200, 64, 64, dtype, seed=62, lens=[200, 7, 130])
    want = check_fwd(x)
    off = lambda t, n: torch.cat([t.new_zeros(n), t.flatten()])[n:].view(t.shape)  # noqa: E731
    n = 16 // x["q"].element_size()
    y = {m: off(x[m], n) for m in ("q", "k", "v")}
    o, C = capi.linattn_fwd(**y, log_decay=off(x["log_decay"], 1), state=off(x["state"], 4), lens=off(x["lens"], 3))
    assert torch.equal(o, want[0]) and torch.equal(C, want[1])
    with pytest.raises(capi.XlstmError):
        capi.linattn_fwd(off(x["q"], 1), x["k"], x["v"], x["log_decay"])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_many_sequences(dtype):
    """More heads than a grid's second axis holds."""
    x = make(70001, 1, 3, 16, 16, dtype, seed=61)
    check_fwd(x)
    check_bwd(x)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_offsets_past_32_bits(dtype):
    """One sequence of more than 2^31 values: its last tokens against 64 bits.  With l = e^-0.5 a token 500 places away
    weighs e^-250, nothing beside the bound's absolute part."""
    T, dqk, dv, N = (1 << 22) + 77, 16, 512, 600
    q, k = (normal(1, 1, T, dqk, dtype=dtype, seed=70 + i) for i in range(2))
    v = normal(1, 1, T, dv, dtype=dtype, seed=72)
    ld = torch.tensor([-0.5], device="cuda")
    o, C = capi.linattn_fwd(q, k, v, ld)
    end = [t[:, :, -N:].contiguous() for t in (q, k, v)]
    want, mag = (f(*end, ld, scale=0.25) for f in (ref.fwd, ref.fwd_magnitude))
    near(o[:, :, -100:], want[0][:, :, -100:], ref.output_bound(want[0], mag[0], N, dqk, dtype)[:, :, -100:], "o")
    near(C, want[1], ref.state_bound(mag[1], N, 0, dtype), "C")
    g = capi.linattn_bwd(q, k, v, ld, o)
    want, mag = (f(*end, ld, o[:, :, -N:], scale=0.25) for f in (ref.bwd, ref.bwd_magnitude))
    for n in ("dq", "dk", "dv"):
        near(g[n][:, :, -100:], want[n][:, :, -100:], ref.output_bound(want[n], mag[n], N, dv, dtype)[:, :, -100:], n)
    o, C = capi.linattn_step(*(normal(8200, 1, d, dtype=dtype, seed=75) for d in (512, 512, 512)), ld,
                             big := normal(8200, 1, 512, 512, seed=76))
    o1, C1 = capi.linattn_step(*(normal(8200, 1, d, dtype=dtype, seed=75)[-2:] for d in (512, 512, 512)), ld, big[-2:])
    assert torch.equal(o[-2:], o1) and torch.equal(C[-2:], C1)


@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_norm_offsets_past_32_bits(layout):
    T, D, N = (1 << 21) + 5, 512, 40
    x = normal(1, 2, T, D, dtype=BF16, seed=80) if layout == "heads" else normal(1, T, 2, D, dtype=BF16, seed=80)
    gate, dy = normal(1, T, 2 * D, dtype=BF16, seed=81), normal(1, T, 2 * D, dtype=BF16, seed=82)
    end = x[:, :, -N:] if layout == "heads" else x[:, -N:]
    small = dict(gate=gate[:, -N:].contiguous(), layout=layout)
    y, g = capi.group_norm(x, gate=gate, layout=layout), capi.group_norm_bwd(dy, x, gate=gate, layout=layout)
    y1 = capi.group_norm(end.contiguous(), **small)
    g1 = capi.group_norm_bwd(dy[:, -N:].contiguous(), end.contiguous(), **small)
    assert torch.equal(y[:, -N:], y1) and torch.equal(g["dgate"][:, -N:], g1["dgate"])
    assert torch.equal(g["dx"][:, :, -N:] if layout == "heads" else g["dx"][:, -N:], g1["dx"])
