"""The operators of a model with recurrent attention state, as they are measured: linear attention
with a decay per head (prompt, single token, gradient), beam search's selection over beams and
vocabulary, and the reordering of prefix states that follows it.

Shapes are those of the library: q [B, Hq, T, 64], k and v [B, Hkv, T, 64], Hq / Hkv <= 8,
14 query heads over 2 key/value heads being its usual layer.  Formulas:

  prefill      S_t = l S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  l = exp(log_decay[kv head])
  step         the same for one token
  backward     gradients of prefill in q, k, v and the first state
  select       the n best of scores[b, i] + log_softmax(logits[b, i])[t] over (i, t)
  decode_beam  one token of the positive-quadratic attention on the states of chosen parents
  reorder      the states of chosen parents, copied to new places
"""
import math

import torch

own = False  # True: the framework's kernels; False: elementary torch operations

D = 64              # head dimension of q, k and v
CHUNK = 128         # tokens per chunk of the plain form
FEATURES, FEATURES_PAD = 2145, 2176   # rows of a packed positive-quadratic state
HEADER_BYTES = 256
UNIT = FEATURES_PAD * (D + 1)         # floats of one (sequence, kv head) of that state
PAD_TOKEN = 1       # the token that an ended beam goes on with


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # a short prompt of one user: latency counts
        dict(name="prefill short", op="prefill", B=1, T=100, Hq=14, Hkv=2, dtype="bf16",
             ragged=False, state=False),
        # the library's usual layer: one prompt of 4096 tokens, 14/2 heads
        dict(name="prefill 4096", op="prefill", B=1, T=4096, Hq=14, Hkv=2, dtype="bf16",
             ragged=False, state=False),
        # a padded batch of prompts of different lengths that go on from a held state
        dict(name="prefill padded batch", op="prefill", B=8, T=4096, Hq=14, Hkv=2, dtype="bf16",
             ragged=True, state=True),
        # full precision, as many key/value heads as query heads, an odd length
        dict(name="prefill fp32", op="prefill", B=2, T=1001, Hq=8, Hkv=8, dtype="fp32",
             ragged=False, state=True),
        # one training sequence of the usual layer
        dict(name="backward 4096", op="backward", B=1, T=4096, Hq=14, Hkv=2, dtype="bf16",
             ragged=False, state=False),
        # a full-precision gradient through a carried state, ragged
        dict(name="backward fp32", op="backward", B=2, T=777, Hq=6, Hkv=3, dtype="fp32",
             ragged=True, state=True),
        # serving: one token for each of 64 sequences
        dict(name="step 64", op="step", B=64, Hq=14, Hkv=2, dtype="bf16"),
        # serving: a full card of sequences, as many key/value heads as query heads
        dict(name="step 1024", op="step", B=1024, Hq=16, Hkv=16, dtype="bf16"),
        # one user's beam search over a small vocabulary: latency counts
        dict(name="select 1x4", op="select", B=1, beams=4, V=32000, n=4, dtype="fp32",
             finished=False),
        # a batch of searches over a large vocabulary, twice the beams kept, some ended
        dict(name="select 16x8", op="select", B=16, beams=8, V=151936, n=16, dtype="bf16",
             finished=True),
        # the beam search's decode step at batch 64 (16 searches of 4 beams)
        dict(name="decode of 16x4 beams", op="decode_beam", B=16, beams=4, Hq=14, Hkv=2,
             dtype="bf16"),
        # the reordering of a small search's states by itself
        dict(name="reorder 2x4", op="reorder", B=2, beams=4, Hq=14, Hkv=2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv = rng.choice((1, 2, 3, 4, 8))
    return hkv * rng.randint(1, 8 if hkv <= 2 else 16 // hkv), hkv


def draw(rng):
    op = rng.choice(("prefill", "prefill", "backward", "step", "select", "decode_beam", "reorder"))
    if op in ("prefill", "backward"):
        dtype = rng.choice(("bf16", "bf16", "fp32"))
        hq, hkv = _heads(rng)
        t = _log_int(rng, 1, 12000)
        most = (8 * 4096 * 14 if op == "prefill" else 4096 * 14) // (1 if dtype == "bf16" else 8)
        t = max(1, min(t, most // hq))
        b = rng.randint(1, max(1, min(16, most // (hq * t))))
        return dict(op=op, B=b, T=t, Hq=hq, Hkv=hkv, dtype=dtype, ragged=rng.random() < 0.4,
                    state=rng.random() < 0.5)
    if op == "step":
        hq, hkv = _heads(rng)
        return dict(op=op, B=_log_int(rng, 1, 1024), Hq=hq, Hkv=hkv,
                    dtype=rng.choice(("bf16", "fp32")))
    beams = rng.randint(1, 16)
    if op == "select":
        v = _log_int(rng, 100, 260000)
        b = max(1, min(_log_int(rng, 1, 64), 16 * 8 * 151936 // (beams * v)))
        return dict(op=op, B=b, beams=beams, V=v, n=rng.randint(1, 2 * beams),
                    dtype=rng.choice(("bf16", "fp32")), finished=rng.random() < 0.5)
    hq, hkv = _heads(rng)
    b = max(1, min(_log_int(rng, 1, 32), 128 // (beams * hkv)))
    if op == "reorder":
        return dict(op=op, B=b, beams=beams, Hq=hq, Hkv=hkv)
    return dict(op=op, B=b, beams=beams, Hq=hq, Hkv=hkv, dtype=rng.choice(("bf16", "fp32")))


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """Tokens of each sequence of a padded batch (the first is full)."""
    b, t = case["B"], case["T"]
    return [t - (i * t) // b if case["ragged"] else t for i in range(b)]


# ---- inputs --------------------------------------------------------------------------------
def _pairs(dev):
    """(r, t) of each packed row of a positive-quadratic state, in its documented order."""
    r, t = [], []
    for a in range(8):
        for b in range(a + 1, 8):
            r += [8 * a + x for x in range(8) for _ in range(8)]
            t += [8 * b + y for _ in range(8) for y in range(8)]
    for a in range(8):
        r += [8 * a + x for x in range(8) for _ in range(x, 8)]
        t += [8 * a + y for x in range(8) for y in range(x, 8)]
    return (torch.tensor(r + list(range(64)) + [64], device=dev),
            torch.tensor(t + [64] * 65, device=dev))


def _state_bytes(b, hq, hkv):
    return HEADER_BYTES + (hq * FEATURES_PAD * 4 + 255) // 256 * 256 + b * hkv * UNIT * 4


def _units(buf, b, hq, hkv):
    """The sums of a state buffer: [B * Hkv][2176 * 64 values, then 2176 normalisers]."""
    return buf[_state_bytes(0, hq, hkv):].view(torch.float32).view(b * hkv, UNIT)


def _quadratic_state(b, hq, hkv, gen, dev, pairs):
    """A prefix state in the library's documented layout: header, readout coefficients of each
    query head (8 groups of dimensions, eps 1e-3) and the sums over 256 tokens."""
    buf = torch.zeros(_state_bytes(b, hq, hkv), dtype=torch.uint8, device=dev)
    head = torch.tensor([0x534C414F, 1, b, hq, hkv, D, D, FEATURES_PAD], dtype=torch.int32)
    buf[:32] = head.view(torch.uint8).to(dev)
    buf[32:40] = torch.tensor([256], dtype=torch.int64).view(torch.uint8).to(dev)
    buf[40:44] = torch.tensor([1e-3], dtype=torch.float32).view(torch.uint8).to(dev)
    r, t = pairs
    n = 8
    L = torch.randn(hq, n + 1, n + 1, generator=gen, device=dev).tril() * 0.3
    L.diagonal(dim1=1, dim2=2).abs_().add_(0.3)
    M = L @ L.transpose(1, 2)
    group = torch.randint(1, n + 1, (hq, 64), generator=gen, device=dev)
    group = torch.cat([group, torch.zeros(hq, 1, dtype=group.dtype, device=dev)], 1)
    s = torch.full((65,), 0.125, device=dev)
    s[64] = 1.0
    coef = M[torch.arange(hq, device=dev)[:, None], group[:, r], group[:, t]]
    coef = coef * torch.where(r == t, 1.0, 2.0) * s[r] * s[t]
    coef[:, FEATURES - 1] += 1e-3
    c = buf[HEADER_BYTES:HEADER_BYTES + hq * FEATURES_PAD * 4].view(torch.float32)
    c.view(hq, FEATURES_PAD)[:, :FEATURES] = coef
    units = _units(buf, b, hq, hkv)
    one = torch.ones(hkv, 256, 1, device=dev)
    for i in range(b):
        k1 = torch.cat([torch.randn(hkv, 256, 64, generator=gen, device=dev), one], 2)
        v1 = torch.cat([torch.randn(hkv, 256, 64, generator=gen, device=dev), one], 2)
        sums = (k1[:, :, r] * k1[:, :, t]).transpose(1, 2) @ v1
        units[i * hkv:(i + 1) * hkv, :FEATURES * D] = sums[:, :, :D].reshape(hkv, -1)
        units[i * hkv:(i + 1) * hkv, FEATURES_PAD * D:FEATURES_PAD * D + FEATURES] = sums[:, :, D]
    return buf


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    op = case["op"]
    st = dict(case)
    if op in ("prefill", "backward", "step"):
        t = 1 if op == "step" else case["T"]
        b, hq, hkv, dt = case["B"], case["Hq"], case["Hkv"], _type(case)
        st.update(q=randn(b, hq, t, D).to(dt), k=randn(b, hkv, t, D).to(dt),
                  v=randn(b, hkv, t, D).to(dt), scale=D ** -0.5)
        # decays 1 - 2^-1 ... 1 - 2^-10, as retention layers spread them over their heads
        st["log_decay"] = torch.log1p(-torch.exp2(
            -1.0 - 9.0 * torch.rand(hkv, generator=gen, device=dev)))
        if op == "step":
            st["state"] = randn(b, hkv, D, D)
            return st
        st["lens"] = (torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
                      if case["ragged"] else None)
        st["state"] = randn(b, hkv, D, D) if case["state"] else None
        # rows behind a sequence's end keep what is there
        if op == "backward":
            st["dout"] = randn(b, hq, t, D).to(dt)
            st["dstate"] = randn(b, hkv, D, D) if case["state"] else None
            st["grads"] = [torch.zeros(b, h, t, D, dtype=dt, device=dev) for h in (hq, hkv, hkv)]
        else:
            st["out"] = torch.zeros(b, hq, t, D, dtype=dt, device=dev)
        if own:  # the scratch memory that a program keeps from call to call
            from positive_quadratic_b200 import oal
            st["workspace"] = (oal.decay_prefill_workspace if op == "prefill" else
                               oal.decay_backward_workspace)(st["q"], st["k"], st["v"])
    elif op == "select":
        b, m, v = case["B"], case["beams"], case["V"]
        st["logits"] = (3.0 * randn(b, m, v)).to(_type(case))
        st["running"] = -20.0 * torch.rand(b, m, generator=gen, device=dev)
        st["ended"] = (torch.rand(b, m, generator=gen, device=dev) < 0.2).to(torch.uint8) \
            if case["finished"] else None
        if own:
            from positive_quadratic_b200 import oal
            st["workspace"] = oal.beam_select_workspace(b, m, v, case["n"], dev)
    else:
        rows, hq, hkv = case["B"] * case["beams"], case["Hq"], case["Hkv"]
        st["pairs"] = _pairs(dev)
        st["src"] = _quadratic_state(rows, hq, hkv, gen, dev, st["pairs"])
        st["dst"] = torch.zeros_like(st["src"])
        # parents within each search, some chosen several times and some not at all
        st["parents"] = (torch.randint(0, case["beams"], (case["B"], case["beams"]),
                                       generator=gen, device=dev)
                         + case["beams"] * torch.arange(case["B"], device=dev)[:, None]
                         ).to(torch.int32)
        if op == "decode_beam":
            dt = _type(case)
            st.update(q=randn(rows, hq, 1, D).to(dt), k=randn(rows, hkv, 1, D).to(dt),
                      v=randn(rows, hkv, 1, D).to(dt))
            if own:
                from positive_quadratic_b200 import oal
                st["workspace"] = oal.decode_workspace(rows, hq, hkv, dev)
    return st


# ---- one pass ------------------------------------------------------------------------------
def run(st):
    return (_run_own if own else _run_plain)[st["op"]](st)


def _state_outputs(st):
    buf = st["dst"]
    coef = buf[HEADER_BYTES:HEADER_BYTES + st["Hq"] * FEATURES_PAD * 4].view(torch.float32)
    return {"tokens": buf[32:40].view(torch.int64), "coef": coef,
            "sums": _units(buf, st["B"] * st["beams"], st["Hq"], st["Hkv"])}


def _own_prefill(st):
    from positive_quadratic_b200 import oal
    args = (st["q"], st["k"], st["v"], st["log_decay"], st["scale"])
    keep = dict(lens=st["lens"], out=st["out"], workspace=st["workspace"])
    if st["state"] is None:
        out, state = oal.decay_prefill(*args, **keep)
        return {"out": out, "state": state}
    out = oal.decay_prefill_continue(*args, st["state"], **keep)
    return {"out": out, "state": st["state"]}


def _own_backward(st):
    from positive_quadratic_b200 import oal
    return oal.decay_backward(st["q"], st["k"], st["v"], st["log_decay"], st["scale"],
                              st["dout"], lens=st["lens"], state=st["state"],
                              dlast=st["dstate"], grads=st["grads"], workspace=st["workspace"])


def _own_step(st):
    from positive_quadratic_b200 import oal
    out = oal.decay_step(st["q"], st["k"], st["v"], st["log_decay"], st["scale"], st["state"])
    return {"out": out, "state": st["state"]}


def _own_select(st):
    from positive_quadratic_b200 import oal
    scores, parents, tokens = oal.beam_select(st["logits"], st["running"], st["n"],
                                              ended=st["ended"], pad_token=PAD_TOKEN,
                                              workspace=st["workspace"])
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _own_decode_beam(st):
    from positive_quadratic_b200 import oal
    out = oal.decode_step_beam(st["q"], st["k"], st["v"], st["src"], st["parents"], st["dst"],
                               st["workspace"])
    return {"out": out, **_state_outputs(st)}


def _own_reorder(st):
    from positive_quadratic_b200 import oal
    oal.state_reorder(st["src"], st["parents"], st["dst"], st["Hq"], st["Hkv"])
    return _state_outputs(st)


_run_own = dict(prefill=_own_prefill, backward=_own_backward, step=_own_step, select=_own_select,
                decode_beam=_own_decode_beam, reorder=_own_reorder)


def _mix(x, y, z, g, first):
    """U_i = sum_{j <= i} l^(i-j) (x_i . y_j) z_j + l^(i+1) x_i first, [B, H, T, D], in chunks:
    products within a chunk, and the sums of earlier chunks carried to it by powers of l."""
    b, h, t, d = x.shape
    n = (t + CHUNK - 1) // CHUNK
    cut = lambda a: torch.nn.functional.pad(a, (0, 0, 0, n * CHUNK - t)).view(  # noqa: E731
        b, h, n, CHUNK, d)
    x, y, z = cut(x), cut(y), cut(z)
    g = g.view(1, h, 1, 1, 1)
    i = torch.arange(CHUNK, device=x.device, dtype=g.dtype)
    apart = i[:, None] - i[None, :]
    within = torch.where(apart >= 0, torch.exp(g * apart.clamp(min=0)), 0.0)
    u = ((x @ y.transpose(3, 4)) * within) @ z
    own_sum = (y * torch.exp(g * (CHUNK - 1 - i)[:, None])).transpose(3, 4) @ z
    c = torch.arange(n, device=x.device, dtype=g.dtype)
    steps = c[:, None] - 1 - c[None, :]
    carry = torch.where(steps >= 0, torch.exp(g[:, :, 0] * CHUNK * steps.clamp(min=0)), 0.0)
    before = (carry @ own_sum.view(b, h, n, d * d)).view(b, h, n, d, d)
    if first is not None:
        before = before + torch.exp(g * CHUNK * c[:, None, None]) * first[:, :, None]
    u = u + torch.exp(g * (i + 1)[:, None]) * (x @ before)
    return u.reshape(b, h, n * CHUNK, d)[:, :, :t]


def _sums(y, z, g, power):
    """sum_j l^power_j y_j z_j^T over the tokens whose power is not negative; power [B, T]."""
    p = power[:, None]
    w = torch.where(p >= 0, torch.exp(g[None, :, None].double() * p.clamp(min=0)), 0.0)
    return (y * w.to(y.dtype)[..., None]).transpose(2, 3) @ z


def _faded(state, g, n):
    return state * torch.exp(g[None, :].double() * n[:, None])[..., None, None].float()


def _valid(st):
    """(mask [B, 1, T, 1] of the tokens that count, lengths [B])."""
    b, t, dev = st["B"], st["T"], st["q"].device
    n = st["lens"].long() if st["lens"] is not None else torch.full((b,), t, device=dev)
    return (torch.arange(t, device=dev)[None, :] < n[:, None])[:, None, :, None], n


def _plain_prefill(st):
    group = st["Hq"] // st["Hkv"]
    mask, n = _valid(st)
    q, k, v = (torch.where(mask, st[x].float(), 0.0) for x in "qkv")
    g, first = st["log_decay"], st["state"]
    wide = lambda a: a.repeat_interleave(group, 1)  # noqa: E731
    u = _mix(q, wide(k), wide(v), g.repeat_interleave(group),
             None if first is None else wide(first))
    out = torch.where(mask, (st["scale"] * u).to(st["out"].dtype), st["out"])
    state = _sums(k, v, g, n[:, None] - 1 - torch.arange(st["T"], device=q.device)[None, :])
    if first is not None:
        state = first.copy_(state + _faded(first, g, n))
    return {"out": out, "state": state}


def _plain_backward(st):
    b, hq, hkv, t = st["B"], st["Hq"], st["Hkv"], st["T"]
    group = hq // hkv
    mask, n = _valid(st)
    q, k, v, do = (torch.where(mask, st[x].float(), 0.0) for x in ("q", "k", "v", "dout"))
    g, scale, first, dlast = st["log_decay"], st["scale"], st["state"], st["dstate"]
    gq = g.repeat_interleave(group)
    wide = lambda a: a.repeat_interleave(group, 1)  # noqa: E731
    shared = lambda a: a.view(b, hkv, group, *a.shape[2:]).sum(2)  # noqa: E731
    back = lambda a: a.flip(2)  # noqa: E731
    dq = scale * _mix(do, wide(v), wide(k), gq,
                      None if first is None else wide(first).transpose(2, 3))
    dk = scale * shared(back(_mix(back(wide(v)), back(do), back(q), gq, None)))
    dv = scale * shared(back(_mix(back(wide(k)), back(q), back(do), gq, None)))
    at = torch.arange(t, device=q.device)[None, :]
    dfirst = scale * shared(_sums(q, do, gq, torch.where(mask[:, 0, :, 0], at + 1, -1)))
    if dlast is not None:
        left = torch.where(mask[:, 0, :, 0], n[:, None] - 1 - at, 0)
        w = torch.exp(g[None, :, None].double() * left[:, None]).float()[..., None]
        dk = dk + w * (v @ dlast.transpose(2, 3))
        dv = dv + w * (k @ dlast)
        dfirst = dfirst + _faded(dlast, g, n)
    dq, dk, dv = (torch.where(mask, x.to(o.dtype), o) for x, o in zip((dq, dk, dv), st["grads"]))
    return {"dq": dq, "dk": dk, "dv": dv, "dstate": dfirst}


def _plain_step(st):
    group = st["Hq"] // st["Hkv"]
    q, k, v = (st[x].float() for x in "qkv")
    decay = torch.exp(st["log_decay"])[None, :, None, None]
    st["state"].copy_(st["state"] * decay + k.transpose(2, 3) @ v)
    out = st["scale"] * (q @ st["state"].repeat_interleave(group, 1))
    return {"out": out.to(_type(st)), "state": st["state"]}


def _plain_select(st):
    # in 64 bits: candidates of different beams may lie next to one another
    x = st["logits"].double()
    b, m, v = x.shape
    top = x.amax(2, keepdim=True)
    logp = x - top - torch.log(torch.exp(x - top).sum(2, keepdim=True))
    if st["ended"] is not None:  # an ended beam goes on with the padding token alone
        pad = torch.where(torch.arange(v, device=x.device) == PAD_TOKEN, 0.0, -math.inf)
        logp = torch.where(st["ended"][:, :, None] != 0, pad, logp)
    flat = (st["running"].double()[:, :, None] + logp).view(b, m * v)
    best, at = torch.sort(flat, dim=1, descending=True, stable=True)
    best, at = best[:, :st["n"]], at[:, :st["n"]]
    row = m * torch.arange(b, device=x.device)[:, None]
    return {"scores": best.float(), "parents": (row + at // v).int(), "tokens": (at % v).int()}


def _plain_reorder(st):
    rows, hq, hkv = st["B"] * st["beams"], st["Hq"], st["Hkv"]
    body = _state_bytes(0, hq, hkv)
    st["dst"][:body] = st["src"][:body]
    src = _units(st["src"], rows, hq, hkv).view(rows, hkv, UNIT)
    _units(st["dst"], rows, hq, hkv).view(rows, hkv, UNIT)[:] = src[st["parents"].view(-1).long()]
    return _state_outputs(st)


def _plain_decode_beam(st):
    rows, hq, hkv = st["B"] * st["beams"], st["Hq"], st["Hkv"]
    group = hq // hkv
    _plain_reorder(st)
    st["dst"][32:40].view(torch.int64).add_(1)
    r, t = st["pairs"]
    one = lambda a: torch.cat([a, torch.ones_like(a[..., :1])], 2)  # noqa: E731
    q, k, v = (one(st[x].float()[:, :, 0]) for x in "qkv")
    units = _units(st["dst"], rows, hq, hkv).view(rows, hkv, UNIT)
    hv = units[:, :, :FEATURES * D].view(rows, hkv, FEATURES, D)
    z = units[:, :, FEATURES_PAD * D:FEATURES_PAD * D + FEATURES]
    psi = k[:, :, r] * k[:, :, t]
    hv += psi[..., None] * v[:, :, None, :D]
    z += psi
    coef = _state_outputs(st)["coef"].view(hq, FEATURES_PAD)[:, :FEATURES]
    phi = (coef * q[:, :, r] * q[:, :, t]).view(rows, hkv, group, FEATURES)
    u, norm = phi @ hv, phi @ z[..., None]
    return {"out": (u / norm).view(rows, hq, 1, D), **_state_outputs(st)}


_run_plain = dict(prefill=_plain_prefill, backward=_plain_backward, step=_plain_step,
                  select=_plain_select, decode_beam=_plain_decode_beam, reorder=_plain_reorder)


# ---- what one pass cannot do without -------------------------------------------------------
def work(case):
    op = case["op"]
    size = 2 if case.get("dtype") == "bf16" else 4
    if op == "select":
        rows = case["B"] * case["beams"]
        # an ended beam's logits need not be read; one beam in five has ended
        live = rows * case["V"] * (0.8 if case["finished"] else 1.0)
        return {"bytes": live * size + 5 * rows + 12 * case["B"] * case["n"], "flops": 4.0 * live}
    hq, hkv = case["Hq"], case["Hkv"]
    if op in ("decode_beam", "reorder"):
        rows, m = case["B"] * case["beams"], case["beams"]
        # each chosen parent is read once; some are chosen twice and some not at all
        read = 1 - (1 - 1 / m) ** m
        moved = rows * hkv * FEATURES * (D + 1) * 4 * (1 + read) + 2 * hq * FEATURES * 4 + 4 * rows
        if op == "reorder":
            return {"bytes": moved, "flops": 0}
        return {"bytes": moved + rows * D * ((hq + 2 * hkv) * size + 4 * hq),
                "flops": 2.0 * rows * FEATURES * (D + 1) * (hq + hkv)}
    b = case["B"]
    state = b * hkv * D * D * 4
    tokens = b if op == "step" else sum(_lengths(case))
    row = D * size * tokens
    one = 2.0 * D * D * tokens
    if op == "step":
        return {"bytes": row * (2 * hq + 2 * hkv) + 2 * state, "flops": one * (hq + hkv)}
    held = state if case["state"] else 0
    if op == "prefill":
        return {"bytes": row * (2 * hq + 2 * hkv) + state + held, "flops": one * (hq + hkv)}
    # q, dout, k, v read and dq, dk, dv written; both states, the first and the last one's gradient
    return {"bytes": row * (3 * hq + 4 * hkv) + state + 2 * held,
            "flops": one * (2 * hq + 3 * hkv)}


# ---- the definitions in 64 bits ------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return dict(prefill=_exact_prefill, backward=_exact_backward, step=_exact_step,
                select=_exact_select, decode_beam=_exact_decode, reorder=_exact_reorder)[
                    case["op"]](st)


def _weights(g, n):
    """l^(i-j) for j <= i, else 0: [n, n], looked up by distance in a table of powers."""
    power = torch.exp(g * torch.arange(n, device=g.device, dtype=torch.float64))
    i = torch.arange(n, device=g.device)
    far = i.view(n, 1) - i.view(1, n)
    return power[far.abs()].masked_fill_(far < 0, 0.0)


def _exact_prefill(st):
    group, scale = st["Hq"] // st["Hkv"], st["scale"]
    out = st["out"].double().clone()
    state = torch.zeros(st["B"], st["Hkv"], D, D, dtype=torch.float64, device=out.device)
    for b, n in enumerate(_lengths(st)):
        for h in range(st["Hkv"]):
            g = st["log_decay"][h].double()
            k, v = (st[x][b, h, :n].double() for x in "kv")
            W = _weights(g, n)
            first = st["state"][b, h].double() if st["state"] is not None else state[b, h].clone()
            since = torch.exp(g * torch.arange(1, n + 1, device=g.device))[:, None]
            for a in range(h * group, (h + 1) * group):
                q = st["q"][b, a, :n].double()
                out[b, a, :n] = scale * ((W * (q @ k.T)) @ v + since * (q @ first))
            last = torch.exp(g * torch.arange(n - 1, -1, -1, device=g.device))[:, None]
            state[b, h] = torch.exp(g * n) * first + (last * k).T @ v
    return {"out": out, "state": state}


def _exact_backward(st):
    group, scale = st["Hq"] // st["Hkv"], st["scale"]
    dq, dk, dv = (x.double().clone() for x in st["grads"])
    dfirst = torch.zeros(st["B"], st["Hkv"], D, D, dtype=torch.float64, device=dq.device)
    zero = torch.zeros(D, D, dtype=torch.float64, device=dq.device)
    for b, n in enumerate(_lengths(st)):
        for h in range(st["Hkv"]):
            g = st["log_decay"][h].double()
            k, v = (st[x][b, h, :n].double() for x in "kv")
            W = _weights(g, n)
            first = st["state"][b, h].double() if st["state"] is not None else zero
            dlast = st["dstate"][b, h].double() if st["dstate"] is not None else zero
            since = torch.exp(g * torch.arange(1, n + 1, device=g.device))[:, None]
            left = torch.exp(g * torch.arange(n - 1, -1, -1, device=g.device))[:, None]
            dk[b, h, :n] = left * (v @ dlast.T)
            dv[b, h, :n] = left * (k @ dlast)
            dfirst[b, h] = torch.exp(g * n) * dlast
            for a in range(h * group, (h + 1) * group):
                q, do = (st[x][b, a, :n].double() for x in ("q", "dout"))
                P, dP = W * (q @ k.T), W * (do @ v.T)
                dq[b, a, :n] = scale * (dP @ k + since * (do @ first.T))
                dk[b, h, :n] += scale * (dP.T @ q)
                dv[b, h, :n] += scale * (P.T @ do)
                dfirst[b, h] += scale * ((since * q).T @ do)
    return {"dq": dq, "dk": dk, "dv": dv, "dstate": dfirst}


def _exact_step(st):
    group = st["Hq"] // st["Hkv"]
    q, k, v = (st[x][:, :, 0].double() for x in "qkv")
    state = st["state"].double() * st["log_decay"].double().exp().view(1, -1, 1, 1)
    state = state + torch.einsum("bhr,bhc->bhrc", k, v)
    q = q.view(q.shape[0], st["Hkv"], group, D)
    out = st["scale"] * torch.einsum("bhgr,bhrc->bhgc", q, state)
    return {"out": out.reshape(st["B"], st["Hq"], 1, D), "state": state}


def _exact_select(st):
    x = st["logits"].double()
    b, m, v = x.shape
    logp = x - torch.logsumexp(x, 2, keepdim=True)
    if st["ended"] is not None:
        logp[st["ended"].bool()] = torch.tensor([-math.inf], dtype=torch.float64, device=x.device)
        logp[..., PAD_TOKEN] = torch.where(st["ended"].bool(), 0.0, logp[..., PAD_TOKEN])
    total = (logp + st["running"].double()[:, :, None]).view(b, -1)
    least = torch.topk(total, st["n"], 1).values[:, -1:]
    found = []
    for one, low in zip(total, least):  # equal scores in the order of their places
        at = torch.nonzero(one >= low)[:, 0]
        ranked = sorted(zip((-one[at]).tolist(), at.tolist()))[:st["n"]]
        found.append([(-score, place // v, place % v) for score, place in ranked])
    found = torch.tensor(found, dtype=torch.float64, device=x.device)
    row = m * torch.arange(b, device=x.device)[:, None]
    return {"scores": found[..., 0], "parents": found[..., 1].long() + row,
            "tokens": found[..., 2].long()}


def _exact_reorder(st):
    rows, hkv = st["B"] * st["beams"], st["Hkv"]
    base = _state_bytes(0, st["Hq"], hkv)
    coef = st["src"][HEADER_BYTES:HEADER_BYTES + st["Hq"] * FEATURES_PAD * 4].view(torch.float32)
    sums = st["src"][base:].view(torch.float32).view(rows, -1).double()
    sums = torch.index_select(sums, 0, st["parents"].view(-1).long())
    return {"tokens": st["src"][32:40].view(torch.int64), "coef": coef.double(),
            "sums": sums.view(rows * hkv, UNIT)}


def _exact_decode(st):
    rows, hq, hkv = st["B"] * st["beams"], st["Hq"], st["Hkv"]
    got = _exact_reorder(st)
    got["tokens"] = got["tokens"] + 1
    r, t = st["pairs"]
    units = got["sums"].view(rows, hkv, UNIT)
    coef = got["coef"].view(hq, FEATURES_PAD)[:, :FEATURES]
    out = torch.empty(rows, hq, 1, D, dtype=torch.float64, device=units.device)
    one = torch.ones(1, dtype=torch.float64, device=units.device)
    for a in range(rows):
        for h in range(hkv):
            k, v = (torch.cat([st[x][a, h, 0].double(), one]) for x in "kv")
            hv = units[a, h, :FEATURES * D].view(FEATURES, D)
            z = units[a, h, FEATURES_PAD * D:FEATURES_PAD * D + FEATURES]
            hv += torch.outer(k[r] * k[t], v[:D])
            z += k[r] * k[t]
            g = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            q = torch.cat([st["q"][a, g, 0].double(), one.expand(hq // hkv, 1)], 1)
            phi = coef[g] * q[:, r] * q[:, t]
            out[a, g, 0] = (phi @ hv) / (phi @ z)[:, None]
    return {"out": out, **got}
