"""Linear attention with a decay per head on the GPU: prompts, continuation, single tokens and
gradients against a plain 64-bit implementation, and the calls around them."""
import math
import os
import subprocess
import sys

import pytest
import torch

from positive_quadratic_b200 import oal
from tests import _decay_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SCALE = 0.125


def make(cuda, B, T, Hq, Hkv, dtype, seed=0, state=False, decay=None):
    gen = torch.Generator().manual_seed(1000 * seed + 7 * T + 3 * Hq + B)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v, do = (r(B, h, T, 64).to(dtype).to(cuda) for h in (Hq, Hkv, Hkv, Hq))
    g = -torch.exp2(-10 * torch.rand(Hkv, generator=gen)) if decay is None \
        else torch.tensor([decay] * Hkv)
    S, R = (r(B, Hkv, 64, 64).to(cuda) if state else None for _ in range(2))
    return q, k, v, g.float().to(cuda), do, S, R


def clean():
    torch.cuda.synchronize()
    assert oal.device_error() == 0


SHAPES = [(1, 1, 1, 1), (2, 2, 2, 1), (1, 63, 7, 1), (2, 64, 6, 3), (1, 65, 8, 1), (3, 127, 2, 2),
          (1, 128, 14, 2), (2, 129, 4, 4), (1, 255, 3, 1), (2, 300, 14, 2), (1, 1000, 5, 5),
          (1, 2049, 4, 2),
          (1, 1000, 56, 8),   # a group of 7 summed in uneven parts
          (2, 1100, 28, 4)]   # several query heads in a row per block, which share their tiles


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,Hq,Hkv", SHAPES)
def test_prefill(cuda, dtype, B, T, Hq, Hkv):
    q, k, v, g, _, S, _ = make(cuda, B, T, Hq, Hkv, dtype, state=True)
    out, state = oal.decay_prefill(q, k, v, g, SCALE)
    w = ref.forward(q, k, v, g, SCALE)
    ref.check("out", out, w[0], w[2], dtype, T)
    ref.check("state", state, w[1], w[3], F32, T)
    held = S.clone()
    out = oal.decay_prefill_continue(q, k, v, g, SCALE, held)
    w = ref.forward(q, k, v, g, SCALE, state=S)
    ref.check("out continued", out, w[0], w[2], dtype, T)
    ref.check("state continued", held, w[1], w[3], F32, T)
    clean()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("decay", [0.0, -1e-5, -0.02, -1.0, -8.0, -200.0, -math.inf])
def test_prefill_decays(cuda, dtype, decay):
    q, k, v, g, _, S, _ = make(cuda, 1, 321, 2, 1, dtype, state=True, decay=decay)
    out = oal.decay_prefill_continue(q, k, v, g, SCALE, held := S.clone())
    w = ref.forward(q, k, v, g, SCALE, state=S)
    ref.check("out", out, w[0], w[2], dtype, 321)
    ref.check("state", held, w[1], w[3], F32, 321)
    clean()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_padded_batch(cuda, dtype):
    """Lengths 0 to T; what lies behind them may be NaN or infinite, and rows behind them keep
    what they held."""
    T, lens = 260, [260, 0, 1, 64, 127, 128, 129, 200]
    q, k, v, g, do, S, R = make(cuda, len(lens), T, 4, 2, dtype, state=True)
    for b, n in enumerate(lens):
        for x in (q, k, v, do):
            x[b, :, n:] = math.nan
            x[b, :, n + 1::2] = math.inf
    ln = torch.tensor(lens, dtype=torch.int32, device=cuda)
    out = torch.full_like(q, 3.0)
    held = S.clone()
    oal.decay_prefill_continue(q, k, v, g, SCALE, held, lens=ln, out=out)
    w = ref.forward(q, k, v, g, SCALE, lens=lens, state=S)
    ref.check("out", out, w[0], w[2], dtype, T)
    ref.check("state", held, w[1], w[3], F32, T)
    grads = [torch.full_like(x, 3.0) for x in (q, k, v)]
    got = oal.decay_backward(q, k, v, g, SCALE, do, lens=ln, state=S, dlast=R, grads=grads)
    w = ref.backward(q, k, v, g, SCALE, do, lens=lens, state=S, dlast=R)
    for n, (x, size) in w.items():
        ref.check(n, got[n], x, size, F32 if n == "dstate" else dtype, T)
    for x in (out, *grads):
        for b, n in enumerate(lens):
            assert bool((x[b, :, n:] == 3.0).all())
    fresh, state = oal.decay_prefill(q, k, v, g, SCALE, lens=ln)
    assert bool((fresh[1] == 0).all()) and bool((state[1] == 0).all())
    clean()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_padded_batch_of_many(cuda, dtype):
    """70 sequences of all lengths, runs of empty ones among them."""
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 401, (70,), generator=gen)
    lens[5:44] = 0
    lens[[0, 69]] = 0
    lens[50] = 400
    q, k, v, g, do, S, R = make(cuda, 70, 400, 14, 2, dtype, state=True)
    ln = lens.to(torch.int32).to(cuda)
    held = S.clone()
    out = oal.decay_prefill_continue(q, k, v, g, SCALE, held, lens=ln)
    w = ref.forward(q, k, v, g, SCALE, lens=lens, state=S)
    ref.check("out", out, w[0], w[2], dtype, 400)
    ref.check("state", held, w[1], w[3], F32, 400)
    got = oal.decay_backward(q, k, v, g, SCALE, do, lens=ln, state=S, dlast=R)
    w = ref.backward(q, k, v, g, SCALE, do, lens=lens, state=S, dlast=R)
    for n, (x, size) in w.items():
        ref.check(n, got[n], x, size, F32 if n == "dstate" else dtype, 400)
    none = torch.zeros_like(ln)
    out, state = oal.decay_prefill(q, k, v, g, SCALE, lens=none)
    assert bool((out == 0).all()) and bool((state == 0).all())
    clean()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,Hq,Hkv", SHAPES)
def test_backward(cuda, dtype, B, T, Hq, Hkv):
    q, k, v, g, do, S, R = make(cuda, B, T, Hq, Hkv, dtype, state=True)
    for state, dlast in ((None, None), (S, R)):
        got = oal.decay_backward(q, k, v, g, SCALE, do, state=state, dlast=dlast)
        w = ref.backward(q, k, v, g, SCALE, do, state=state, dlast=dlast)
        for n, (x, size) in w.items():
            ref.check(n, got[n], x, size, F32 if n == "dstate" else dtype, T)
    clean()


@pytest.mark.parametrize("decay", [0.0, -0.5, -math.inf])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_backward_decays(cuda, dtype, decay):
    q, k, v, g, do, S, R = make(cuda, 1, 200, 2, 1, dtype, state=True, decay=decay)
    got = oal.decay_backward(q, k, v, g, SCALE, do, state=S, dlast=R)
    w = ref.backward(q, k, v, g, SCALE, do, state=S, dlast=R)
    for n, (x, size) in w.items():
        ref.check(n, got[n], x, size, F32 if n == "dstate" else dtype, 200)
    clean()


def test_backward_against_differences(cuda):
    """The gradient's products with random directions against central differences of the 64-bit
    forward pass.  The loss is cubic in (q, k, v, S_0) jointly, so a central difference at step h
    is off by exactly h^2 times the third-order term; two steps remove it (Richardson), and what is
    left is the fp32 rounding of the gradient, bounded elementwise, and 64-bit rounding / h."""
    q, k, v, g, do, S, R = make(cuda, 2, 150, 4, 2, F32, state=True)
    got = oal.decay_backward(q, k, v, g, SCALE, do, state=S, dlast=R)
    w = ref.backward(q, k, v, g, SCALE, do, state=S, dlast=R)
    gen = torch.Generator().manual_seed(5)
    xs = [x.double().cpu() for x in (q, k, v, S)]
    ds = [torch.randn(x.shape, generator=gen, dtype=torch.float64) for x in xs]

    def loss(h):
        a = [x + h * d for x, d in zip(xs, ds)]
        o, last, _, _ = ref.forward(*a[:3], g, SCALE, state=a[3])
        return float((o * do.double().cpu()).sum() + (last * R.double().cpu()).sum())

    diff = [(loss(h) - loss(-h)) / (2 * h) for h in (1e-2, 5e-3)]
    slope = (4 * diff[1] - diff[0]) / 3
    names = ("dq", "dk", "dv", "dstate")
    along = sum(float((got[n].double().cpu() * d).sum()) for n, d in zip(names, ds))
    tol = sum(float((ref.tolerance(*w[n], F32, 150) * d.abs()).sum()) for n, d in zip(names, ds))
    assert abs(along - slope) <= tol + 1e-9 * abs(loss(0.0)) / 5e-3


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_then_steps(cuda, dtype):
    """A prompt, its continuation and single tokens give what one prompt over all of it gives."""
    B, T, Hq, Hkv = 2, 333, 6, 2
    q, k, v, g, _, _, _ = make(cuda, B, T, Hq, Hkv, dtype)
    w = ref.forward(q, k, v, g, SCALE)
    cut = lambda a, b: [x[:, :, a:b].contiguous() for x in (q, k, v)]  # noqa: E731
    o1, state = oal.decay_prefill(*cut(0, 200), g, SCALE)
    o2 = oal.decay_prefill_continue(*cut(200, 330), g, SCALE, state)
    o3 = [oal.decay_step(*cut(t, t + 1), g, SCALE, state) for t in range(330, 333)]
    ref.check("out", torch.cat([o1, o2, *o3], 2), w[0], w[2], dtype, T)
    ref.check("state", state, w[1], w[3], F32, T)
    clean()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (16, 2), (14, 2), (5, 5)])
@pytest.mark.parametrize("B", [1, 3, 130])
def test_step(cuda, dtype, B, Hq, Hkv):
    q, k, v, g, _, S, _ = make(cuda, B, 1, Hq, Hkv, dtype, state=True)
    state = S.clone()
    out = oal.decay_step(q, k, v, g, SCALE, state)
    w = ref.forward(q, k, v, g, SCALE, state=S)
    ref.check("out", out, w[0], w[2], dtype, 1)
    ref.check("state", state, w[1], w[3], F32, 1)
    # from parents, several of them the same, into another buffer: as after a reordering
    gen = torch.Generator().manual_seed(B)
    par = torch.randint(0, B, (B,), generator=gen).to(torch.int32).to(cuda)
    dst = torch.full_like(S, math.nan)
    out2 = oal.decay_step(q, k, v, g, SCALE, dst, src=S, parents=par)
    moved = torch.full_like(S, math.nan)
    oal.decay_state_reorder(S, par, moved)
    assert torch.equal(moved, S[par.long()])
    out3 = oal.decay_step(q, k, v, g, SCALE, moved)
    assert torch.equal(out2, out3) and torch.equal(dst, moved)
    clean()


def test_step_spreads_one_state_over_beams(cuda):
    q, k, v, g, _, S, _ = make(cuda, 1, 1, 2, 1, F32, state=True)
    wide = [x.expand(4, -1, -1, -1).contiguous() for x in (q, k, v)]
    dst = torch.empty(4, 1, 64, 64, device=cuda)
    par = torch.zeros(4, dtype=torch.int32, device=cuda)
    out = oal.decay_step(*wide, g, SCALE, dst, src=S, parents=par)
    one = oal.decay_step(q, k, v, g, SCALE, S)
    assert all(torch.equal(out[i], one[0]) and torch.equal(dst[i], S[0]) for i in range(4))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_state_alone_and_empty_prompts(cuda, dtype):
    q, k, v, g, _, S, _ = make(cuda, 2, 140, 4, 2, dtype, state=True)
    _, full = oal.decay_prefill(q, k, v, g, SCALE)
    none, alone = oal.decay_prefill(q, k, v, g, SCALE, want_out=False)
    assert none is None and torch.equal(full, alone)
    e = [x[:, :, :0].contiguous() for x in (q, k, v)]
    _, zero = oal.decay_prefill(*e, g, SCALE, state=torch.full_like(S, 7.0))
    assert bool((zero == 0).all())
    held = S.clone()
    oal.decay_prefill_continue(*e, g, SCALE, held)
    assert torch.equal(held, S)
    got = oal.decay_backward(*e, g, SCALE, e[0], dlast=S)
    assert torch.equal(got["dstate"], S)  # no token: the gradient passes through
    nothing = [x[:0].contiguous() for x in (q, k, v)]
    out, state = oal.decay_prefill(*nothing, g, SCALE)
    assert out.numel() == 0 and state.numel() == 0
    clean()


def test_bad_values_reach_the_error_word(cuda):
    q, k, v, g, _, S, _ = make(cuda, 2, 70, 2, 1, F32, state=True)
    for bad in (0.5, math.nan, math.inf):
        out, _ = oal.decay_prefill(q, k, v, torch.full_like(g, bad), SCALE)
        assert oal.device_error() == -10
        w = ref.forward(q, k, v, torch.zeros_like(g), SCALE)
        ref.check("counted as 0", out, w[0], w[2], F32, 70)
    for n in (-1, 71):
        ln = torch.tensor([70, n], dtype=torch.int32, device=cuda)
        _, state = oal.decay_prefill(q, k, v, g, SCALE, lens=ln)
        assert oal.device_error() == -10
        w = ref.forward(q, k, v, g, SCALE, lens=[70, min(max(n, 0), 70)])
        ref.check("clamped", state, w[1], w[3], F32, 70)
    par = torch.tensor([5, -3], dtype=torch.int32, device=cuda)
    dst = torch.empty_like(S)
    oal.decay_state_reorder(S, par, dst)
    assert oal.device_error() == -10
    assert torch.equal(dst[0], S[1]) and torch.equal(dst[1], S[0])
    clean()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_repeats_streams_and_graphs(cuda, dtype):
    """The same bits again, on another stream, and from captured graphs that share a workspace and
    are replayed in turn on new inputs."""
    q, k, v, g, do, S, R = make(cuda, 2, 400, 6, 2, dtype, state=True)
    first = oal.decay_prefill(q, k, v, g, SCALE)
    grads = oal.decay_backward(q, k, v, g, SCALE, do, state=S, dlast=R)
    again = oal.decay_prefill(q, k, v, g, SCALE)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = oal.decay_prefill(q, k, v, g, SCALE, stream=side)
    there_g = oal.decay_backward(q, k, v, g, SCALE, do, state=S, dlast=R, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, there))
    assert all(torch.equal(grads[n], there_g[n]) for n in grads)
    ws = oal.decay_backward_workspace(q, k, v)
    ins = [x.clone() for x in (q, k, v, do)]
    A, G = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(A):
        out, state = oal.decay_prefill(*ins[:3], g, SCALE, workspace=ws)
        oal.decay_step(*[x[:, :, :1].contiguous() for x in ins[:3]], g, SCALE, state)
    with torch.cuda.graph(G):
        gg = oal.decay_backward(*ins[:3], g, SCALE, ins[3], state=S, dlast=R, workspace=ws)
    for seed in (1, 2):
        new = make(cuda, 2, 400, 6, 2, dtype, seed=seed)
        for x, y in zip(ins, (*new[:3], new[4])):
            x.copy_(y)
        A.replay()
        G.replay()
        A.replay()
        o, s = oal.decay_prefill(*new[:3], g, SCALE)
        oal.decay_step(*[x[:, :, :1].contiguous() for x in new[:3]], g, SCALE, s)
        w = oal.decay_backward(*new[:3], g, SCALE, new[4], state=S, dlast=R)
        assert torch.equal(out, o) and torch.equal(state, s)
        assert all(torch.equal(gg[n], w[n]) for n in w)
    clean()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_prompt(cuda, dtype):
    """20,001 tokens, sampled rows: the last state and the rows around chunk borders, from the
    definition."""
    T = 20001
    q, k, v, g, _, _, _ = make(cuda, 1, T, 2, 1, dtype, decay=-1e-3)
    out, state = oal.decay_prefill(q, k, v, g, SCALE)
    qd, kd, vd = (x.double().cpu() for x in (q, k, v))
    for i in (0, 127, 128, 6399, 6400, 12345, 20000):
        w = torch.exp(-1e-3 * torch.arange(i, -1, -1).double())
        for h in range(2):
            s = w * (kd[0, 0, :i + 1] @ qd[0, h, i])
            want = SCALE * (s @ vd[0, 0, :i + 1])
            size = SCALE * (w * (kd[0, 0, :i + 1].abs() @ qd[0, h, i].abs())) @ vd[
                0, 0, :i + 1].abs()
            ref.check(f"row {i}", out[0, h, i], want, size, dtype, T)
    w = torch.exp(-1e-3 * torch.arange(T - 1, -1, -1).double())[:, None]
    ref.check("state", state[0, 0], (w * kd[0, 0]).T @ vd[0, 0],
              (w * kd[0, 0].abs()).T @ vd[0, 0].abs(), F32, T)


def test_first_call_inside_a_capture(cuda):
    """A process whose first call is captured: nothing of the call's set-up breaks the capture."""
    code = """
import torch
from positive_quadratic_b200 import oal
torch.manual_seed(0)
q, k, v = (torch.randn(1, h, 300, 64, device="cuda").bfloat16() for h in (2, 1, 1))
g, ws = torch.full((1,), -0.1, device="cuda"), torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
x, run = torch.randn(1, 2, 5000, device="cuda"), torch.zeros(1, 2, device="cuda")
torch.cuda.synchronize()
G = torch.cuda.CUDAGraph()
with torch.cuda.graph(G):
    out, state = oal.decay_prefill(q, k, v, g, 0.125, workspace=ws)
    best = oal.beam_select(x, run, 4, workspace=ws[1 << 21:])
    dq = oal.decay_backward(q, k, v, g, 0.125, out, workspace=ws)["dq"]
G.replay()
o, s = oal.decay_prefill(q, k, v, g, 0.125)
assert torch.equal(out, o) and torch.equal(state, s)
assert torch.equal(dq, oal.decay_backward(q, k, v, g, 0.125, out)["dq"])
assert all(torch.equal(a, b) for a, b in zip(best, oal.beam_select(x, run, 4)))
assert oal.device_error() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True, timeout=300)


def test_two_streams_at_once(cuda):
    """Calls on two streams with workspaces of their own do not disturb one another."""
    a = make(cuda, 2, 700, 14, 2, BF, seed=1)
    b = make(cuda, 1, 900, 4, 4, BF, seed=2)
    want = [oal.decay_prefill(*x[:3], x[3], SCALE) for x in (a, b)]
    grads = [oal.decay_backward(*x[:3], x[3], SCALE, x[4]) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got, got_g = [], []
    for _ in range(5):
        for x, s in zip((a, b), streams):
            got.append(oal.decay_prefill(*x[:3], x[3], SCALE, stream=s))
            got_g.append(oal.decay_backward(*x[:3], x[3], SCALE, x[4], stream=s))
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(got, got_g)):
        assert all(torch.equal(p, q) for p, q in zip(x, want[i % 2]))
        assert all(torch.equal(y[n], grads[i % 2][n]) for n in y)
    clean()


def test_binding_refusals(cuda):
    q, k, v, g, do, S, R = make(cuda, 2, 10, 4, 2, BF, state=True)
    ok = lambda **kw: oal.decay_prefill(**{**dict(  # noqa: E731
        q=q, k=k, v=v, log_decay=g, scale=SCALE), **kw})
    ok()
    for bad in (dict(k=k.float()), dict(log_decay=g.double()), dict(q=q.half()),
                dict(lens=torch.zeros(2, dtype=torch.int64, device=cuda)), dict(out=q.float()),
                dict(state=S.bfloat16())):
        with pytest.raises(TypeError):
            ok(**bad)
    for bad in (dict(k=k[:, :, :9].contiguous()), dict(v=v[:1].contiguous()), dict(log_decay=g[:1]),
                dict(q=q.transpose(1, 2)), dict(k=k.cpu()), dict(out=q[:, :2]), dict(state=S[:1]),
                dict(lens=torch.zeros(3, dtype=torch.int32, device=cuda)),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(oal.OALError):  # heads that do not divide, another head dimension
        oal.decay_prefill(q[:, :3].contiguous(), k, v, g, SCALE)
    with pytest.raises(oal.OALError):
        oal.decay_prefill(*[x[..., :32].contiguous() for x in (q, k, v)], g, SCALE)
    with pytest.raises(oal.OALError):
        ok(workspace=torch.empty(256, dtype=torch.uint8, device=cuda))
    with pytest.raises(ValueError):
        oal.decay_prefill_continue(q, k, v, g, SCALE, None)
    one = [x[:, :, :1].contiguous() for x in (q, k, v)]
    par = torch.zeros(2, dtype=torch.int32, device=cuda)
    for args in (dict(src=S), dict(parents=par), dict(src=S, parents=par[:1]),
                 dict(src=S[..., :32].contiguous(), parents=par)):
        with pytest.raises(ValueError):
            oal.decay_step(*one, g, SCALE, R, **args)
    with pytest.raises(oal.OALError):  # in place through parents
        oal.decay_step(*one, g, SCALE, S, src=S, parents=par)
    with pytest.raises(ValueError):
        oal.decay_step(q, k, v, g, SCALE, S)
    with pytest.raises(TypeError):
        oal.decay_backward(q, k, v, g, SCALE, do.float())
    clean()
