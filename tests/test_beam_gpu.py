"""Beam search on recurrent state: the selection against a plain 64-bit one, the copies of states
bit for bit, and a whole search."""
import math

import numpy as np
import pytest
import torch

from positive_quadratic_b200 import inputs, oal
from tests import _decay_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def plain_select(logits, running, n, ended=None, pad=0):
    """The definition: every candidate's score in 64 bits, sorted by (-score, place)."""
    x = logits.double().cpu().numpy()
    run = running.double().cpu().numpy()
    B, m, V = x.shape
    scores, parents, tokens = (np.zeros((B, n)) for _ in range(3))
    for b in range(B):
        s = np.full((m, V), -np.inf)
        for i in range(m):
            if not np.isfinite(run[b, i]):
                continue
            if ended is not None and bool(ended[b, i]):
                s[i, pad] = run[b, i]
                continue
            top = x[b, i].max()
            if not np.isfinite(top):  # NaN, +inf or nothing finite
                continue
            s[i] = run[b, i] + (x[b, i] - top - np.log(np.exp(x[b, i] - top).sum()))
        flat = s.reshape(-1)
        at = np.lexsort((np.arange(flat.size), -flat))[:n]
        scores[b], parents[b], tokens[b] = flat[at], b * m + at // V, at % V
    return scores, parents.astype(int), tokens.astype(int)


def check_select(logits, running, n, ended=None, pad=0):
    got = oal.beam_select(logits, running, n, ended=ended, pad_token=pad)
    s, p, t = (x.cpu().numpy() for x in got)
    ws, wp, wt = plain_select(logits, running, n, ended, pad)
    assert (p == wp).all() and (t == wt).all()
    live = np.isfinite(ws)
    assert (np.isneginf(s) == ~live).all()
    # lse: exponentials good to 2^-20 relative (2 units of the approximation and the rounding of
    # x - top and of its product), so lse to 2^-20; the score is rounded once
    tol = 2.0 ** -20 + 2.0 ** -24 * np.abs(ws[live])
    assert (np.abs(s[live] - ws[live]) <= tol).all()
    torch.cuda.synchronize()
    assert oal.device_error() == 0


def make(cuda, B, beams, V, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + V + beams)
    x = (3 * torch.randn(B, beams, V, generator=gen)).to(dtype).to(cuda)
    return x, (-20 * torch.rand(B, beams, generator=gen)).to(cuda)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,beams,V,n", [
    (1, 1, 1, 1), (2, 1, 5, 5), (1, 2, 3, 6), (3, 4, 100, 8), (2, 4, 1000, 4), (1, 4, 1024, 32),
    (2, 3, 1025, 6), (1, 1, 2047, 32), (1, 2, 2048, 3), (2, 2, 2049, 17), (1, 8, 8191, 16),
    (1, 4, 8193, 9), (2, 16, 16385, 32), (1, 256, 50, 32), (1, 2, 1000003, 32), (70, 1, 33, 2), (1, 5, 50257, 10), (40, 8, 50257, 16), (3, 1, 131072, 1)])
def test_select(cuda, dtype, B, beams, V, n):
    check_select(*make(cuda, B, beams, V, dtype), n)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [8185, 8187, 8189, 16381])
def test_select_in_a_made_workspace(cuda, dtype, V):
    """One workspace serves logits of either type, at lengths where theirs differ too."""
    x, run = make(cuda, 2, 3, V, dtype)
    ws = oal.beam_select_workspace(2, 3, V, 5, cuda)
    got = oal.beam_select(x, run, 5, workspace=ws)
    _, parents, tokens = plain_select(x, run, 5)
    assert (got[1].cpu().numpy() == parents).all() and (got[2].cpu().numpy() == tokens).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [7, 1500, 9001, 70000])
def test_select_ties(cuda, dtype, V):
    """Equal logits (all of them, and a few values over and over) in the order of their places;
    equal rows in the order of the rows; zeros of either sign are equal."""
    x, run = make(cuda, 2, 3, V, dtype)
    same = torch.zeros_like(x)
    check_select(same, run, 9)
    check_select(same, torch.zeros_like(run), 9)
    few = torch.randint(0, 3, x.shape, generator=torch.Generator().manual_seed(V)).to(x)
    check_select(few, torch.zeros_like(run), 21)
    signed = torch.where(few > 1, -0.0, 0.0).to(dtype)
    check_select(signed, torch.zeros_like(run), 5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [40, 3000, 20000])
def test_select_masks(cuda, dtype, V):
    """Masked logits (-inf, and the type's lowest value), rows with nothing left, NaN and +inf."""
    x, run = make(cuda, 2, 6, V, dtype)
    x[0, 0] = -math.inf                      # nothing left
    x[0, 1, 3:] = -math.inf                  # three left
    x[0, 2] = torch.finfo(dtype).min         # all at the lowest value: a uniform row
    x[0, 3, 5] = math.nan
    x[0, 4, V - 1] = math.inf
    x[0, 5, : V - 2] = torch.finfo(dtype).min
    x[1, :, 1:] = -math.inf                  # one token in each of six rows
    check_select(x, run, 8)
    check_select(x[:, :2].contiguous(), run[:, :2].contiguous(), 16)
    run[1, 0] = -math.inf
    run[1, 1] = math.nan
    run[1, 2] = math.inf
    check_select(x, run, 8)
    first = torch.full_like(run, -math.inf)  # a search's first step: one row counts
    first[:, 0] = 0
    check_select(make(cuda, 2, 6, V, dtype)[0], first, 6)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pad", [0, 2, 99])
def test_select_ended_rows(cuda, dtype, pad):
    x, run = make(cuda, 3, 4, 100, dtype)
    ended = torch.tensor([[1, 0, 0, 1], [0, 0, 0, 0], [1, 1, 1, 1]], dtype=torch.uint8, device=cuda)
    x[0, 0] = math.nan  # not read
    check_select(x, run, 8, ended, pad)
    check_select(x, run, 8, ended.bool(), pad)
    run[2, 1] = -math.inf
    check_select(x, run, 3, ended, pad)


def test_select_spaced_rows_streams_and_graphs(cuda):
    wide, run = make(cuda, 2, 3, 1024, BF)
    check_select(wide[:, :, :1001], run, 7)
    x, run = make(cuda, 4, 4, 9000, F32)
    ws = oal.beam_select_workspace(4, 4, 9000, 8, cuda)
    want = oal.beam_select(x, run, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = oal.beam_select(x, run, 8, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    G = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(G):
        got = oal.beam_select(xs, run, 8, workspace=ws)
    for seed in (1, 2):
        y, _ = make(cuda, 4, 4, 9000, F32, seed)
        xs.copy_(y)
        G.replay()
        assert all(torch.equal(a, b) for a, b in zip(oal.beam_select(y, run, 8), got))


def quadratic_state(cuda, B, Hq, Hkv, T=40, dtype="bf16", seed=3):
    p = inputs.small_layer(seed, B=B, T=T, Hq=Hq, Hkv=Hkv, dtype=dtype)
    t = lambda a, d=None: torch.from_numpy(np.ascontiguousarray(a)).to(cuda, d)  # noqa: E731
    dt = BF if dtype == "bf16" else F32
    q, k, v = (t(x, dt) for x in (p.q, p.k, p.v))
    _, state = oal.prefill(q, k, v, t(p.group_id), t(p.L), t(p.G), p.eps, 128)
    return state, q, k, v


@pytest.mark.parametrize("B,n,Hq,Hkv", [(1, 4, 14, 2), (6, 6, 4, 4), (8, 3, 8, 1)])
def test_state_reorder(cuda, B, n, Hq, Hkv):
    src, *_ = quadratic_state(cuda, B, Hq, Hkv)
    par = torch.randint(0, B, (n,), generator=torch.Generator().manual_seed(n)).to(
        torch.int32).to(cuda)
    size = oal.state_bytes(oal.make_shape(n, 1, Hq, Hkv))
    dst = torch.full((size,), 0xAB, dtype=torch.uint8, device=cuda)
    oal.state_reorder(src, par, dst, Hq, Hkv)
    head = oal.state_bytes(oal.make_shape(0, 1, Hq, Hkv))
    assert torch.equal(dst[head:].view(n, -1), src[head:].view(B, -1)[par.long()])
    got, want = dst[:32].view(torch.int32).tolist(), src[:32].view(torch.int32).tolist()
    assert got == want[:2] + [n] + want[3:]
    assert torch.equal(dst[32:head], src[32:head])
    torch.cuda.synchronize()
    assert oal.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,n,Hq,Hkv", [(1, 4, 14, 2), (6, 6, 4, 4), (8, 3, 8, 1), (5, 40, 3, 1)])
def test_decode_step_beam(cuda, dtype, B, n, Hq, Hkv):
    """The step from parents equals the reordering followed by the step, bit for bit."""
    src, *_ = quadratic_state(cuda, B, Hq, Hkv, dtype=dtype)
    gen = torch.Generator().manual_seed(n)
    par = torch.randint(0, B, (n,), generator=gen).to(torch.int32).to(cuda)
    dt = BF if dtype == "bf16" else F32
    q, k, v = (torch.randn(n, h, 1, 64, generator=gen).to(dt).to(cuda) for h in (Hq, Hkv, Hkv))
    size = oal.state_bytes(oal.make_shape(n, 1, Hq, Hkv))
    one, two = (torch.full((size,), 0xAB, dtype=torch.uint8, device=cuda) for _ in range(2))
    ws = oal.decode_workspace(n, Hq, Hkv, cuda)
    before = src.clone()
    out = oal.decode_step_beam(q, k, v, src, par, one, ws)
    oal.state_reorder(src, par, two, Hq, Hkv)
    want = oal.decode_step(q, k, v, two, ws)
    assert torch.equal(out, want) and torch.equal(one, two) and torch.equal(src, before)
    torch.cuda.synchronize()
    assert oal.device_error() == 0


def test_decode_step_beam_of_no_sequence(cuda):
    """dst becomes the empty state that the reordering and the step leave."""
    src, *_ = quadratic_state(cuda, 2, 4, 2)
    par = torch.empty(0, dtype=torch.int32, device=cuda)
    q, k = (torch.empty(0, h, 1, 64, dtype=BF, device=cuda) for h in (4, 2))
    size = oal.state_bytes(oal.make_shape(0, 1, 4, 2))
    one, two = (torch.full((size,), 0xAB, dtype=torch.uint8, device=cuda) for _ in range(2))
    ws = oal.decode_workspace(1, 4, 2, cuda)
    oal.decode_step_beam(q, k, k, src, par, one, ws)
    oal.state_reorder(src, par, two, 4, 2)
    assert torch.equal(one, two) and (one != 0xAB).any()


def test_bad_parents_reach_the_error_word(cuda):
    src, *_ = quadratic_state(cuda, 2, 2, 1)
    par = torch.tensor([7, -1], dtype=torch.int32, device=cuda)
    want = torch.empty_like(src)
    oal.state_reorder(src, torch.tensor([1, 0], dtype=torch.int32, device=cuda), want, 2, 1)
    got = torch.empty_like(src)
    oal.state_reorder(src, par, got, 2, 1)
    assert oal.device_error() == -10 and torch.equal(got, want)
    q, k, v = (torch.ones(2, h, 1, 64, device=cuda) for h in (2, 1, 1))
    ws = oal.decode_workspace(2, 2, 1, cuda)
    o1 = oal.decode_step_beam(q, k, v, src, par, got, ws)
    assert oal.device_error() == -10
    o2 = oal.decode_step(q, k, v, want, ws)
    assert torch.equal(o1, o2) and torch.equal(got, want)


@pytest.mark.parametrize("kind", ["decay", "quadratic"])
def test_beam_search(cuda, kind):
    """A prompt, its state spread over the beams, and five steps of select and beam step.  At
    every step the selection equals the plain one on the same logits; at the end every beam's
    state and output are those of its own tokens run from the prompt's state in one line."""
    searches, beams, V, Hq, Hkv, T, steps = 2, 3, 500, 4, 2, 70, 5
    rows = searches * beams
    gen = torch.Generator().manual_seed(11)
    table = [torch.randn(V, h, 64, generator=gen).to(cuda) for h in (Hq, Hkv, Hkv)]
    head = (torch.randn(Hq * 64, V, generator=gen) / 8).to(cuda)
    g = torch.tensor([-0.1, -0.01], device=cuda)
    embed = lambda tok: [t[tok.long().view(-1)][:, :, None].contiguous() for t in table]  # noqa
    if kind == "decay":
        prompt = [torch.randn(searches, h, T, 64, generator=gen).to(cuda) for h in (Hq, Hkv, Hkv)]
        out, state = oal.decay_prefill(*prompt, g, 0.125)
        start = state.clone()
        step = lambda x, src, par: (lambda dst: (oal.decay_step(  # noqa: E731
            *x, g, 0.125, dst, src=src, parents=par), dst))(
                torch.empty(par.numel(), Hkv, 64, 64, device=cuda))
    else:
        state, q, k, v = quadratic_state(cuda, searches, Hq, Hkv, T=T, dtype="fp32")
        start = state.clone()
        out = torch.randn(searches, Hq, T, 64, generator=gen).to(cuda)
        size = oal.state_bytes(oal.make_shape(rows, 1, Hq, Hkv))
        ws = oal.decode_workspace(rows, Hq, Hkv, cuda)
        step = lambda x, src, par: (lambda dst: (oal.decode_step_beam(  # noqa: E731
            *x, src, par, dst, ws), dst))(torch.empty(size, dtype=torch.uint8, device=cuda))
    logits = (out[:, :, -1].reshape(searches, 1, -1) @ head)
    running = torch.zeros(searches, 1, device=cuda)
    origin = list(range(searches))
    history = None
    for s in range(steps):
        run, par, tok = oal.beam_select(logits, running, beams)
        want = plain_select(logits, running, beams)
        assert (par.cpu().numpy() == want[1]).all() and (tok.cpu().numpy() == want[2]).all()
        parents, tokens = par.view(-1).tolist(), tok.view(-1).tolist()
        history = [(history[p] if history else [origin[p]]) + [t] for p, t in zip(parents, tokens)]
        out, state = step(embed(tok), state, par)
        logits = (out.view(searches, beams, -1) @ head)
        running = run
    # each beam by itself
    for r in range(rows):
        who, line = history[r][0], history[r][1:]
        par = torch.full((rows,), who, dtype=torch.int32, device=cuda)
        src = start
        for t in line:
            o, src = step(embed(torch.full((rows,), t, device=cuda)), src, par)
            par = torch.arange(rows, dtype=torch.int32, device=cuda)
        assert torch.equal(o[0], out[r])
        if kind == "decay":
            assert torch.equal(src[0], state[r])
        else:
            base = oal.state_bytes(oal.make_shape(0, 1, Hq, Hkv))
            assert torch.equal(src[base:].view(rows, -1)[0], state[base:].view(rows, -1)[r])
    if kind == "decay":  # and from the definition
        who, line = history[0][0], history[0][1:]
        x = [torch.cat([p[who:who + 1], t[torch.tensor(line, device=cuda)].transpose(0, 1)[None]],
                       2) for p, t in zip(prompt, table)]
        w = _decay_ref.forward(*x, g, 0.125)
        _decay_ref.check("out", out[:1, :, 0], w[0][:, :, -1], w[2][:, :, -1], F32, T + steps)
        _decay_ref.check("state", state[:1], w[1], w[3], F32, T + steps)
    torch.cuda.synchronize()
    assert oal.device_error() == 0


def test_select_of_many_ended_rows(cuda):
    """256 rows, all but a few ended: their padding tokens compete by their running scores."""
    x, run = make(cuda, 2, 256, 300, F32)
    ended = torch.ones(2, 256, dtype=torch.uint8, device=cuda)
    ended[0, 7] = ended[0, 250] = 0
    check_select(x, run, 32, ended, 299)
    check_select(torch.zeros_like(x), torch.zeros_like(run), 32, ended, 3)


def test_select_ties_across_rows_and_tiles(cuda):
    """Thousands of candidates that share the n-th score, in several rows and tiles."""
    x = torch.zeros(1, 4, 40000, device=cuda)
    x[:, :, ::7] = 2.0
    x[0, 2, 39999] = 3.0
    x[0, 0, 5] = 2.5
    run = torch.tensor([[0.0, 0.0, 1.0, 1.0]], device=cuda)
    check_select(x, run, 32)
    check_select(x.bfloat16(), run, 20)
    x[0, 1] = x[0, 0]  # two equal rows
    check_select(x, run, 32)


def test_binding_refusals(cuda):
    x, run = make(cuda, 2, 3, 100, F32)
    for bad in (lambda: oal.beam_select(x.half(), run, 2), lambda: oal.beam_select(x, run.double(), 2),
                lambda: oal.beam_select(x, run, 2, ended=run)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: oal.beam_select(x[0], run, 2), lambda: oal.beam_select(x, run[:, :2], 2),
                lambda: oal.beam_select(x.transpose(1, 2), run, 2),
                lambda: oal.beam_select(x[:, ::2], run[:, ::2].contiguous(), 2, tokens=run),
                lambda: oal.beam_select(x[:, :2], run[:, :2].contiguous(), 2)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (dict(n=33), dict(n=0), dict(n=2, ended=torch.ones(2, 3, dtype=torch.uint8, device=cuda),
                                            pad_token=100)):
        with pytest.raises(oal.OALError):
            oal.beam_select(x, run, **bad)
    with pytest.raises(oal.OALError):  # the rows of a misaligned view
        oal.beam_select(x[:, :, 1:], run, 2)
    src, *_ = quadratic_state(cuda, 2, 2, 1)
    par = torch.zeros(2, dtype=torch.int32, device=cuda)
    for bad in (lambda: oal.state_reorder(src, par, src[:-16], 2, 1),
                lambda: oal.state_reorder(src[:1000], par, src, 2, 1),
                lambda: oal.state_reorder(src, par, src.clone().cpu(), 2, 1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        oal.state_reorder(src, par.long(), src.clone(), 2, 1)
    with pytest.raises(oal.OALError):
        oal.state_reorder(src, par, src, 2, 1)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [1, 7, 1001, 9001, 50257, 250002])
@pytest.mark.parametrize("gap", [0, 1, 6])
def test_select_equal_rows(cuda, dtype, V, gap):
    """Rows of equal logits and running scores tie for every token, wherever they start in memory
    (V + gap is no multiple of a 16-byte vector), and n cuts through a tie."""
    wide = torch.zeros(2, 5, V + gap, dtype=dtype, device=cuda)
    x = wide[:, :, :V]
    x.copy_(make(cuda, 2, 1, V, dtype)[0].expand(2, 5, V))
    x[:, 2] = make(cuda, 2, 1, V, dtype, seed=1)[0][:, 0]
    run = torch.tensor([[-3.3] * 5, [-0.7, -0.7, -9.0, -0.7, -0.7]], device=cuda)
    for n in (2, 6, 11):
        if n <= 5 * V:
            check_select(x, run, n)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("beams", [1, 3, 5])
def test_select_of_rows_that_end_inside_a_vector(cuda, dtype, beams):
    """The array's last vector holds tokens of one row or two, of one tile or two."""
    for V in [*range(1, 12), *range(8185, 8200), *range(16384, 16392)]:
        check_select(*make(cuda, 1, beams, V, dtype), min(4, beams * V))


def test_parents_in_a_larger_buffer(cuda):
    """A buffer with room for eight sequences that holds four: a fifth one is an error of the
    caller's, not what lies there."""
    Hq, Hkv = 4, 2
    src, *_ = quadratic_state(cuda, 4, Hq, Hkv)
    fp32, *_ = quadratic_state(cuda, 4, Hq, Hkv, dtype="fp32")
    for state in (src, fp32):
        assert state[8:12].view(torch.int32).tolist() == [4]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    size = lambda n: oal.state_bytes(oal.make_shape(n, 1, Hq, Hkv))  # noqa: E731
    wide = torch.full((size(8),), 0xAB, dtype=torch.uint8, device=cuda)
    oal.state_reorder(src, i32(0, 1, 2, 3), wide, Hq, Hkv)
    got, want = (torch.empty(size(3), dtype=torch.uint8, device=cuda) for _ in range(2))
    oal.state_reorder(src, i32(3, 0, 2), want, Hq, Hkv)
    oal.state_reorder(wide, i32(3, 0, 2), got, Hq, Hkv)
    torch.cuda.synchronize()
    assert oal.device_error() == 0 and torch.equal(got, want)
    oal.state_reorder(wide, i32(5, -1, 2), got, Hq, Hkv)
    assert oal.device_error() == -10 and torch.equal(got, want)
    gen = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(3, h, 1, 64, generator=gen).to(cuda) for h in (Hq, Hkv, Hkv))
    ws = oal.decode_workspace(3, Hq, Hkv, cuda)
    one = oal.decode_step_beam(q, k, v, wide, i32(4, 0, 2), got, ws)
    assert oal.device_error() == -10
    two = oal.decode_step(q, k, v, want, ws)
    assert torch.equal(one, two) and torch.equal(got, want)
