"""Plain 64-bit linear attention with a decay per key/value head, its gradient by the formulas,
and the error bounds that its kernels are held to.  Written from the definition
o_i = scale sum_{j<=i} l^(i-j) (q_i . k_j) v_j + scale l^(i+1) S_0^T q_i, without chunks."""
import torch


def _powers(g, n):
    """l^(i-j) for j <= i, else 0 (l^0 = 1 for any l)."""
    i = torch.arange(n)
    far = (i[:, None] - i[None, :]).double()
    w = torch.exp(g * far.clamp(min=0))
    return torch.where(far > 0, w, torch.where(far == 0, 1.0, 0.0))


def _since(g, lo, hi, step=1):
    m = torch.arange(lo, hi, step).double()
    return torch.where(m == 0, 1.0, torch.exp(g * m.clamp(min=1)))[:, None]


def _clean(log_decay):
    return torch.clamp(log_decay.double().cpu(), min=-1e4)


def forward(q, k, v, log_decay, scale, lens=None, state=None):
    """(out, last state, bound of out, bound of the state): the bounds are the same sums with the
    magnitudes of every factor.  Rows behind a sequence's end are NaN in out."""
    q, k, v = (x.detach().double().cpu() for x in (q, k, v))
    g = _clean(log_decay)
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    grp = Hq // Hkv
    out, size, near = (torch.full_like(q, float("nan")) for _ in range(3))
    last = torch.zeros(B, Hkv, D, D, dtype=torch.float64)
    last_size = torch.zeros_like(last)
    for b in range(B):
        n = T if lens is None else int(lens[b])
        for h in range(Hkv):
            S0 = torch.zeros(D, D, dtype=torch.float64) if state is None \
                else state[b, h].double().cpu()
            kk, vv = k[b, h, :n], v[b, h, :n]
            W, s1 = _powers(g[h], n), _since(g[h], 1, n + 1)
            for a in range(h * grp, (h + 1) * grp):
                x = q[b, a, :n]
                P = W * (x @ kk.T)
                out[b, a, :n] = scale * (P @ vv + s1 * (x @ S0))
                near[b, a, :n] = abs(scale) * (P.abs() @ vv.abs())
                size[b, a, :n] = abs(scale) * ((W * (x.abs() @ kk.abs().T)) @ vv.abs()
                                               + s1 * (x.abs() @ S0.abs()))
            left = _since(g[h], n - 1, -1, -1)
            all_ = torch.exp(g[h] * n) if n else torch.tensor(1.0).double()
            last[b, h] = all_ * S0 + (left * kk).T @ vv
            last_size[b, h] = all_ * S0.abs() + (left * kk.abs()).T @ vv.abs()
    return out, last, size, last_size


def backward(q, k, v, log_decay, scale, dout, lens=None, state=None, dlast=None):
    """{name: (gradient, bound)} by the formulas."""
    q, k, v, do = (x.detach().double().cpu() for x in (q, k, v, dout))
    g = _clean(log_decay)
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    grp = Hq // Hkv
    res = {n: [torch.full_like(x, float("nan")) for _ in range(2)]
           for n, x in (("dq", q), ("dk", k), ("dv", v))}
    res["dstate"] = [torch.zeros(B, Hkv, D, D, dtype=torch.float64) for _ in range(2)]
    zero = torch.zeros(D, D, dtype=torch.float64)
    for size in (0, 1):
        f = torch.abs if size else (lambda x: x)
        sc = abs(scale) if size else scale
        for b in range(B):
            n = T if lens is None else int(lens[b])
            for h in range(Hkv):
                S0 = f(zero if state is None else state[b, h].double().cpu())
                R = f(zero if dlast is None else dlast[b, h].double().cpu())
                kk, vv = f(k[b, h, :n]), f(v[b, h, :n])
                W, s1 = _powers(g[h], n), _since(g[h], 1, n + 1)
                left = _since(g[h], n - 1, -1, -1)
                dk, dv = left * (vv @ R.T), left * (kk @ R)
                ds = (torch.exp(g[h] * n) if n else 1.0) * R
                for a in range(h * grp, (h + 1) * grp):
                    x, y = f(q[b, a, :n]), f(do[b, a, :n])
                    P, dP = W * (x @ kk.T), W * (y @ vv.T)
                    res["dq"][size][b, a, :n] = sc * (dP @ kk + s1 * (y @ S0.T))
                    dk = dk + sc * dP.T @ x
                    dv = dv + sc * P.T @ y
                    ds = ds + sc * (s1 * x).T @ y
                res["dk"][size][b, h, :n], res["dv"][size][b, h, :n] = dk, dv
                res["dstate"][size][b, h] = ds
    return {n: tuple(x) for n, x in res.items()}


def tolerance(value, size, dtype, T):
    """How far a kernel's value may be off, elementwise.

    fp32: every product and partial sum is rounded to 2^-24 of its own size.  A value is a sum over
    at most 64 dimensions, 128 tokens of a chunk per head of the group, and one term per chunk
    (T / 64 of them); with the powers of l (good to 4 roundings) and the last factors each term
    meets fewer than 300 + T / 64 roundings, so the error is below that many 2^-24 of `size`, the
    sum of the magnitudes.  (8 heads of a group add up to 8 times 128 terms: 1024.)
    bf16: the scores of a chunk and the states before it are rounded once to bf16 (each term off by
    at most 2^-8 of itself), and the result once more.
    """
    few = (300 + 1024 + T / 64) * 2.0 ** -24
    if dtype == torch.float32:
        return few * size + 1e-30
    half = 2.0 ** -8
    return half * value.abs() + (half * (1 + half) + few) * size + 1e-30


def check(name, got, want, size, dtype, T):
    """`got` against (want, size); NaN in want marks what is not compared."""
    got = got.detach().double().cpu()
    live = ~torch.isnan(want)
    err = (got - want).abs()[live]
    tol = tolerance(want, size, dtype, T)[live]
    assert torch.isfinite(got[live]).all(), name
    worst = float((err / tol).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{name}: error is {worst:.2f} times its bound"
