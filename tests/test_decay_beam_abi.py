"""Host-side checks of decayed linear attention, beam selection and state reordering: every refusal
comes before the device is touched, so these run without a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from positive_quadratic_b200 import build, oal

NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE, OVERLAP = -1, -2, -3, -4, -8, -11
BIG = ctypes.c_size_t(1 << 60)
SCALE = ctypes.c_float(0.125)


@pytest.fixture(scope="module")
def L():
    build.build()
    return oal.lib()


def P(addr=1 << 20):
    return ctypes.c_void_p(addr)


def shape(B=2, T=100, Hq=4, Hkv=2, dtype=oal.OAL_BF16, **kw):
    s = oal.make_shape(B, T, Hq, Hkv, 128, dtype)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def size_of(L, fn, s):
    n = ctypes.c_size_t()
    rc = getattr(L, fn)(ctypes.byref(s), ctypes.byref(n))
    return rc, n.value


def test_state_and_workspace_sizes(L):
    assert size_of(L, "oal_decay_state_bytes", shape()) == (0, 2 * 2 * 64 * 64 * 4)
    # fp32: the chunk states, in place; bf16: the chunk sums and the bf16 states before them
    for T, c64, c128 in ((1, 1, 1), (64, 1, 1), (65, 2, 1), (1000, 16, 8)):
        rc, n = size_of(L, "oal_decay_prefill_workspace_bytes", shape(T=T, dtype=oal.OAL_F32))
        assert (rc, n) == (0, 4 * c64 * 16384)
        rc, n = size_of(L, "oal_decay_prefill_workspace_bytes", shape(T=T))
        assert (rc, n) == (0, 4 * c128 * (16384 + 8192))
    assert size_of(L, "oal_decay_prefill_workspace_bytes", shape(T=0))[1] >= 256
    # the gradient: both directions; the reverse one in parts where chunks are few (a group of 2:
    # 2 parts), never in empty ones (a group of 7 over 64 chunks: 4 parts of 2)
    assert size_of(L, "oal_decay_backward_workspace_bytes", shape(T=1000)) == (
        0, 4 * 8 * (2 * 8192 + 3 * 16384))
    assert size_of(L, "oal_decay_backward_workspace_bytes", shape(B=1, T=4096, Hq=14)) == (
        0, 64 * (2 * 8192 + 5 * 16384))


@pytest.mark.parametrize("dtype", [oal.OAL_F32, oal.OAL_BF16])
@pytest.mark.parametrize("T", [0, 1, 300])
def test_sizes_of_an_empty_batch(L, T, dtype):
    for fn in ("oal_decay_prefill_workspace_bytes", "oal_decay_backward_workspace_bytes"):
        assert size_of(L, fn, shape(B=0, T=T, dtype=dtype)) == (0, 256)


@pytest.mark.parametrize("field,value,code", [
    ("Hq", 0, SHAPE), ("Hkv", 3, SHAPE), ("B", -1, SHAPE), ("T", -5, SHAPE), ("dh", 32, UNSUPPORTED),
    ("dv", 128, UNSUPPORTED), ("dtype", 7, UNSUPPORTED), ("Hq", 18, UNSUPPORTED),
    ("T", 1 << 30, SHAPE)])
def test_shapes_are_checked(L, field, value, code):
    s = shape(**{field: value})
    for fn in ("oal_decay_prefill_workspace_bytes", "oal_decay_backward_workspace_bytes"):
        assert size_of(L, fn, s)[0] == code
    assert L.oal_decay_prefill(P(), P(), P(), P(), SCALE, None, P(), P(), P(), BIG, ctypes.byref(s),
                               None) == code
    if field != "T":
        assert L.oal_decay_step(P(), P(), P(), P(), SCALE, None, 0, None, P(), P(), ctypes.byref(s),
                                None) == code


def test_grid_limits(L):
    s = shape(B=32768, T=1)  # B * Hq = 131072 blocks in y
    assert size_of(L, "oal_decay_prefill_workspace_bytes", s)[0] == SHAPE
    assert size_of(L, "oal_decay_state_bytes", s)[0] == 0  # a step has no such limit


def call_prefill(L, s, fn="oal_decay_prefill", q=P(), k=P(), v=P(), g=P(), lens=None, out=P(),
                 state=P(), ws=P(), n=BIG):
    return getattr(L, fn)(q, k, v, g, SCALE, lens, out, state, ws, n, ctypes.byref(s), None)


@pytest.mark.parametrize("dtype", [oal.OAL_F32, oal.OAL_BF16])
def test_prefill_arguments(L, dtype):
    s = shape(dtype=dtype)
    for fn in ("oal_decay_prefill", "oal_decay_prefill_continue"):
        for name in ("q", "k", "v", "g"):
            assert call_prefill(L, s, fn, **{name: None}) == NULL, name
        for name in ("q", "k", "v", "out", "state", "ws"):
            assert call_prefill(L, s, fn, **{name: P((1 << 20) + 8)}) == ALIGN, name
        for name in ("g", "lens"):
            assert call_prefill(L, s, fn, **{name: P((1 << 20) + 2)}) == ALIGN, name
        assert call_prefill(L, s, fn, ws=None) == WORKSPACE
        assert call_prefill(L, s, fn, n=ctypes.c_size_t(64)) == WORKSPACE
    assert call_prefill(L, s, out=None, state=None) == NULL
    assert call_prefill(L, s, "oal_decay_prefill_continue", state=None) == NULL
    assert L.oal_decay_prefill(P(), P(), P(), P(), SCALE, None, P(), P(), P(), BIG, None, None) == NULL
    # nothing to do: no sequence; no token to continue with
    assert call_prefill(L, shape(B=0, dtype=dtype), q=None, k=None, v=None, out=None, state=None) == 0
    assert call_prefill(L, shape(T=0, dtype=dtype), "oal_decay_prefill_continue", q=None, k=None,
                        v=None, out=None) == 0


def test_backward_arguments(L):
    s = shape()
    names = ("q", "k", "v", "g", "lens", "dout", "state", "dlast", "dq", "dk", "dv", "dstate")

    def call(ws=P(), n=BIG, **kw):
        a = dict.fromkeys(names, P())
        a.update(lens=None, state=None, dlast=None, dstate=None)
        a.update(kw)
        return L.oal_decay_backward(a["q"], a["k"], a["v"], a["g"], SCALE, a["lens"], a["dout"],
                                    a["state"], a["dlast"], a["dq"], a["dk"], a["dv"], a["dstate"], ws,
                                    n, ctypes.byref(s), None)

    for name in ("q", "k", "v", "g", "dout", "dq", "dk", "dv"):
        assert call(**{name: None}) == NULL, name
    for name in names:
        off = 2 if name in ("g", "lens") else 8
        assert call(**{name: P((1 << 20) + off)}) == ALIGN, name
    assert call(ws=None) == WORKSPACE and call(n=ctypes.c_size_t(1 << 10)) == WORKSPACE


def test_step_arguments(L):
    s = shape(T=1)
    size = 2 * 2 * 16384

    def call(q=P(), k=P(), v=P(), g=P(), src=None, n=0, parents=None, state=P(), out=P()):
        return L.oal_decay_step(q, k, v, g, SCALE, src, n, parents, state, out, ctypes.byref(s), None)

    for name in ("q", "k", "v", "g", "state", "out"):
        assert call(**{name: None}) == NULL, name
    for name in ("q", "k", "v", "state", "out"):
        assert call(**{name: P((1 << 20) + 8)}) == ALIGN, name
    far = P((1 << 20) + size)
    assert call(src=far, n=2) == NULL and call(parents=P(), n=2) == NULL  # they go together
    assert call(src=far, n=0, parents=P()) == SHAPE
    assert call(src=P((1 << 20) + size - 16), n=2, parents=P()) == OVERLAP
    assert call(src=P((1 << 20) - size + 16), n=2, parents=P()) == OVERLAP
    assert call(src=P(1 << 20), n=2, parents=P()) == OVERLAP


def select(L, logits=P(), ld=1000, dtype=oal.OAL_BF16, running=P(), ended=None, pad=0, B=2, beams=4,
           V=1000, n=4, scores=P(), parents=P(), tokens=P(), ws=P(), nb=BIG):
    return L.oal_beam_select(logits, ld, dtype, running, ended, pad, B, beams, V, n, scores, parents,
                             tokens, ws, nb, None)


def test_select_arguments(L):
    for kw in (dict(B=-1), dict(beams=0), dict(V=0), dict(n=0), dict(ld=999), dict(beams=1, V=3, n=4, ld=3),
               dict(B=20000), dict(V=(1 << 29) - 1, ld=1 << 30),
               dict(ended=P(), pad=1000), dict(ended=P(), pad=-1)):
        assert select(L, **kw) == SHAPE, kw
    for kw in (dict(n=33), dict(beams=257), dict(dtype=2)):
        assert select(L, **kw) == UNSUPPORTED, kw
    for name in ("logits", "running", "scores", "parents", "tokens"):
        assert select(L, **{name: None}) == NULL, name
        assert select(L, **{name: P((1 << 20) + 2)}) == ALIGN, name
    assert select(L, ws=None) == WORKSPACE and select(L, nb=ctypes.c_size_t(1)) == WORKSPACE
    assert select(L, B=0, logits=None, running=None) == 0
    n = ctypes.c_size_t()
    assert L.oal_beam_select_workspace_bytes(2, 4, 1000, 33, 0, ctypes.byref(n)) == UNSUPPORTED
    assert L.oal_beam_select_workspace_bytes(2, 4, 1000, 4, 0, None) == NULL


def test_largest_vocabularies(L):
    """Places of the last tile count up to two tiles past V, in 32 bits."""
    n = ctypes.c_size_t()
    size = lambda beams, V, dt: L.oal_beam_select_workspace_bytes(  # noqa: E731
        1, beams, V, 1, dt, ctypes.byref(n))
    for dt in (oal.OAL_F32, oal.OAL_BF16):
        assert size(1, (1 << 31) - (1 << 14) - 1, dt) == 0
        assert size(1, (1 << 31) - (1 << 14), dt) == SHAPE
        assert size(1, (1 << 31) - 65, dt) == SHAPE
        assert size(8, (1 << 28) - (1 << 11), dt) == SHAPE


@pytest.mark.parametrize("V", [1, 7, 8185, 8186, 8187, 8189, 8190, 8192, 8195, 16381])
def test_select_workspace_holds_either_type(V):
    """A bf16 row may begin up to 7 logits behind a 16-byte boundary, an fp32 row 3: one tile more
    for some lengths."""
    ws = oal.beam_select_workspace(2, 3, V, 1, "cpu")
    assert all(ws.numel() >= oal._select_bytes(2, 3, V, 1, code)
               for code in (oal.OAL_BF16, oal.OAL_F32))


A, STEP = 1 << 32, 1 << 24  # places far apart


def apart(*names):
    return {name: A + i * STEP for i, name in enumerate(names)}


def ptrs(d):
    return {k: P(v) for k, v in d.items()}


@pytest.mark.parametrize("dtype", [oal.OAL_F32, oal.OAL_BF16])
@pytest.mark.parametrize("fn", ["oal_decay_prefill", "oal_decay_prefill_continue"])
def test_prefill_over_its_inputs(L, fn, dtype):
    s = shape(dtype=dtype)
    at = apart("q", "k", "v", "g", "out", "state", "ws")
    for w in ("out", "state"):
        for r in ("q", "k", "v", "out"):
            if w != r:
                assert call_prefill(L, s, fn, **ptrs({**at, w: at[r]})) == OVERLAP, (w, r)
                assert call_prefill(L, s, fn, **ptrs({**at, w: at[r] + 16})) == OVERLAP, (w, r)


def test_step_over_its_inputs(L):
    s = shape(T=77)  # T is not used: one token
    at = apart("q", "k", "v", "g", "state", "out")
    for w in ("out", "state"):
        for r in ("q", "k", "v", "out"):
            if w != r:
                a = ptrs({**at, w: at[r]})
                assert L.oal_decay_step(a["q"], a["k"], a["v"], a["g"], SCALE, None, 0, None, a["state"],
                                        a["out"], ctypes.byref(s), None) == OVERLAP, (w, r)


def test_backward_over_its_inputs(L):
    s = shape()
    ins, outs = ("q", "k", "v", "dout", "state"), ("dq", "dk", "dv", "dstate")
    at = apart(*ins, *outs, "g", "dlast", "ws")
    for w in outs:
        for r in ins + outs + ("dlast",):
            off = 16 if r == "dlast" else 0  # dlast itself may be dstate
            if w == r or (r == "dlast" and w != "dstate"):
                continue
            a = ptrs({**at, w: at[r] + off})
            assert L.oal_decay_backward(
                a["q"], a["k"], a["v"], a["g"], SCALE, None, a["dout"], a["state"], a["dlast"], a["dq"],
                a["dk"], a["dv"], a["dstate"], a["ws"], BIG, ctypes.byref(s), None) == OVERLAP, (w, r)


def test_select_over_its_inputs(L):
    at = apart("logits", "running", "ended", "scores", "parents", "tokens", "ws")
    for w in ("scores", "parents", "tokens"):
        for r in ("running", "ended", "scores", "parents", "tokens"):
            if w != r:
                assert select(L, **ptrs({**at, w: at[r]})) == OVERLAP, (w, r)


def test_reorder_arguments(L):
    s = shape(B=3)
    size = oal.state_bytes(s)
    a, b = 1 << 30, (1 << 30) + size
    r = lambda src=P(a), n=3, par=P(), dst=P(b), s=s: L.oal_state_reorder(  # noqa: E731
        src, n, par, dst, ctypes.byref(s), None)
    assert r(src=None) == NULL and r(par=None) == NULL and r(dst=None) == NULL
    assert r(n=0) == SHAPE and r(s=shape(B=70000, T=1)) == SHAPE
    assert r(src=P(a + 8)) == ALIGN and r(dst=P(b + 8)) == ALIGN and r(par=P(a + 2)) == ALIGN
    assert r(dst=P(a)) == OVERLAP and r(dst=P(b - 16)) == OVERLAP
    d = lambda src, dst, n=3: L.oal_decay_state_reorder(  # noqa: E731
        src, n, P(), dst, ctypes.byref(s), None)
    rows = 3 * 2 * 16384
    assert d(P(a), P(a + rows - 16)) == OVERLAP and d(None, P(a)) == NULL
    z = shape(B=0)
    assert L.oal_decay_state_reorder(P(a), 3, None, P(b), ctypes.byref(z), None) == 0
    beam = lambda q=P(), src=P(a), n=3, par=P(), dst=P(b), out=P(), ws=P(), nb=BIG: (  # noqa: E731
        L.oal_decode_step_beam(q, P(), P(), src, n, par, dst, out, ws, nb, ctypes.byref(s), None))
    assert beam(q=None) == NULL and beam(par=None) == NULL and beam(out=P(8)) == ALIGN
    assert beam(ws=None) == WORKSPACE and beam(nb=ctypes.c_size_t(16)) == WORKSPACE
    assert beam(dst=P(a + 16)) == OVERLAP and beam(n=0) == SHAPE


def test_binding_refuses_host_tensors():
    q, k = torch.zeros(1, 2, 1, 64), torch.zeros(1, 1, 1, 64)
    g, state = torch.zeros(1), torch.zeros(1, 1, 64, 64)
    i32 = torch.zeros(1, dtype=torch.int32)
    buf = torch.zeros(oal.state_bytes(oal.make_shape(1, 1, 2, 1)), dtype=torch.uint8)
    for call in (lambda: oal.decay_prefill(q, k, k, g, 0.1),
                 lambda: oal.decay_prefill_continue(q, k, k, g, 0.1, state),
                 lambda: oal.decay_step(q, k, k, g, 0.1, state),
                 lambda: oal.decay_step(q=q, k=k, v=k, log_decay=g, scale=0.1, state=state),
                 lambda: oal.decay_backward(q, k, k, g, 0.1, q),
                 lambda: oal.beam_select(torch.zeros(1, 1, 5), torch.zeros(1, 1), 2),
                 lambda: oal.state_reorder(buf, i32, buf.clone(), 2, 1),
                 lambda: oal.decay_state_reorder(state, i32, state.clone()),
                 lambda: oal.decode_step_beam(q, k, k, buf, i32, buf.clone(), buf)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_select_over_its_logits(L):
    """Results anywhere from the first logit of the first row to the last one of the last."""
    at = apart("logits", "running", "ended", "scores", "parents", "tokens", "ws")
    last = at["logits"] + 2 * (7 * 1004 + 1000) - 4  # 8 rows of 1000 bf16, 1004 apart
    for w in ("scores", "parents", "tokens"):
        for place in (at["logits"], at["logits"] + 4000, last, at["logits"] - 4):
            assert select(L, ld=1004, **ptrs({**at, w: place})) == OVERLAP, (w, place)


def test_step_from_parents_over_its_inputs(L):
    s = shape(T=1)
    at = apart("q", "k", "v", "g", "src", "parents", "state", "out")

    def call(**kw):
        a = ptrs({**at, **kw})
        return L.oal_decay_step(a["q"], a["k"], a["v"], a["g"], SCALE, a["src"], 3, a["parents"],
                                a["state"], a["out"], ctypes.byref(s), None)

    last = at["src"] + 3 * 2 * 16384 - 16
    for place in (at["src"], last, at["g"], at["parents"]):
        assert call(out=place) == OVERLAP and call(state=place) == OVERLAP, place


def test_backward_over_the_last_state_gradient(L):
    """Every gradient but dstate, which may be dlast itself; and the decays and lengths."""
    s = shape()
    at = apart("q", "k", "v", "g", "lens", "dout", "state", "dlast", "dq", "dk", "dv", "dstate", "ws")

    def call(**kw):
        a = ptrs({**at, **kw})
        return L.oal_decay_backward(
            a["q"], a["k"], a["v"], a["g"], SCALE, a["lens"], a["dout"], a["state"], a["dlast"],
            a["dq"], a["dk"], a["dv"], a["dstate"], a["ws"], BIG, ctypes.byref(s), None)

    for w in ("dq", "dk", "dv"):
        for place in (at["dlast"], at["dlast"] + 2 * 2 * 16384 - 16):
            assert call(**{w: place}) == OVERLAP, w
    for w in ("dq", "dk", "dv", "dstate"):
        for r in ("g", "lens"):
            assert call(**{w: at[r]}) == OVERLAP, (w, r)
    assert call(dstate=at["dlast"] + 16) == OVERLAP


def test_decode_step_beam_over_its_inputs(L):
    s = shape(B=3, T=1)
    at = apart("q", "k", "v", "src", "parents", "dst", "out", "ws")
    ends = {"src": oal.state_bytes(shape(B=4, T=1)), "dst": oal.state_bytes(s), "q": 3 * 4 * 64 * 2,
            "k": 3 * 2 * 64 * 2, "v": 3 * 2 * 64 * 2}

    def call(**kw):
        a = ptrs({**at, **kw})
        return L.oal_decode_step_beam(a["q"], a["k"], a["v"], a["src"], 4, a["parents"], a["dst"],
                                      a["out"], a["ws"], BIG, ctypes.byref(s), None)

    for r, size in ends.items():
        for place in (at[r], at[r] + size - 16):
            assert call(out=place) == OVERLAP, r
            if r != "dst":
                assert call(dst=place) == OVERLAP, r
    assert call(out=at["parents"]) == OVERLAP and call(dst=at["parents"]) == OVERLAP


@pytest.mark.parametrize("fn", ["oal_decay_prefill", "oal_decay_prefill_continue"])
def test_prefill_over_decays_and_lengths(L, fn):
    at = apart("q", "k", "v", "g", "lens", "out", "state", "ws")
    for w in ("out", "state"):
        for r in ("g", "lens"):
            assert call_prefill(L, shape(), fn, **ptrs({**at, w: at[r]})) == OVERLAP, (w, r)


def test_reorder_over_its_indices(L):
    s = shape(B=3)
    at = ptrs(apart("src", "parents", "dst"))
    for fn in ("oal_state_reorder", "oal_decay_state_reorder"):
        assert getattr(L, fn)(at["src"], 3, at["dst"], at["dst"], ctypes.byref(s), None) == OVERLAP
        inside = P(at["dst"].value + 3 * 2 * 16384 - 4)
        assert getattr(L, fn)(at["src"], 3, inside, at["dst"], ctypes.byref(s), None) == OVERLAP


def test_binding_loads_on_a_torch_without_cuda():
    """Size queries and refusals work there."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from positive_quadratic_b200 import oal
assert oal.state_bytes(oal.make_shape(1, 1, 2, 1)) > 0
x = torch.zeros(1, 1, 1, 64)
try:
    oal.decay_step(x, x, x, torch.zeros(1), 0.1, torch.zeros(1, 1, 64, 64))
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("a host tensor passed")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(oal.__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)


def test_binding_refuses_a_stream_of_another_device():
    """The call would run on another stream than the one named."""
    class There:  # stands for a tensor, or a stream, of a device that is not here
        def __init__(self, index):
            self.index, self.device = index, torch.device("cuda", index)

        def get_device(self):
            return self.index

    ran = []
    call = oal._call_on_stream(lambda x, stream: ran.append(stream))
    with pytest.raises(ValueError, match="stream"):
        call(There(0), stream=There(1))
    assert not ran


@pytest.mark.parametrize("Hq,Hkv", [(0, 0), (2, 0), (0, 1), (-2, -1)])
def test_state_buffers_need_heads(Hq, Hkv):
    with pytest.raises(ValueError, match="Hq"):
        oal._state_of("src", torch.zeros(1 << 16, dtype=torch.uint8), 1, Hq, Hkv, -1)
