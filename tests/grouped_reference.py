"""Plain 64-bit forms of the 16-bit operators (grouped products, combine,
adapters and their gradients) on the CPU, each with an element-wise bound on
what a kernel that multiplies exactly, sums in fp32 and rounds once may be off.

The bound of a stored sum is
    half a step of the stored type  (eps / 2 relative: bf16 2^-8, fp16 2^-11, fp32 2^-24)
  + (terms + 32) 2^-24 sum |products|  (one fp32 rounding per term, and the joins of partial sums)
and, where a factor is itself such a sum, its own bound times the other factor.
fp16 results also get half of fp16's smallest step, 2^-25.
"""
import torch

F8 = torch.float64
U = 2.0 ** -24


def d(t):
    return t.detach().to("cpu").to(F8)


def stored(value, slack, dtype):
    """Bound of `value` known within `slack`, once it is rounded to dtype."""
    half = torch.finfo(dtype).eps / 2
    return half * (value.abs() + slack) + slack + (2.0 ** -25 if dtype == torch.float16 else 0.0) + 1e-300


def sums(terms, magnitude):
    return (terms + 32) * U * magnitude


def within(got, value, bound, what=""):
    got = d(got)
    assert got.shape == value.shape, (what, got.shape, value.shape)
    if value.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - value).abs() - bound
    worst = over.argmax()
    assert over.max() <= 0, (what, "off by", float((got - value).abs().flatten()[worst]), "allowed", float(bound.flatten()[worst]),
                             "value", float(value.flatten()[worst]), "at", int(worst))


def gather(A, a_row, P):
    """Rows row(p) of A; a row outside A is zeros."""
    A = d(A)
    at = torch.arange(P) if a_row is None else a_row.cpu().long()
    ok = (at >= 0) & (at < A.shape[0])
    rows = A[torch.where(ok, at, 0)] if A.shape[0] else torch.zeros((P, A.shape[1]), dtype=F8)
    return torch.where(ok[:, None], rows, 0.0)


def spans(offsets):
    o = offsets.cpu().tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def grouped(A, W, offsets, a_row, P):
    """(C, sum of |products|, rows that belong to a group)."""
    x, W = gather(A, a_row, P), d(W)
    C, M = (torch.zeros((P, W.shape[1]), dtype=F8) for _ in range(2))
    used = torch.zeros(P, dtype=torch.bool)
    for e, a, b in spans(offsets):
        C[a:b] = x[a:b] @ W[e].T
        M[a:b] = x[a:b].abs() @ W[e].abs().T
        used[a:b] = True
    return C, M, used


def grouped_dgrad(dC, W, offsets):
    dC, W = d(dC), d(W)
    D, M = (torch.zeros((dC.shape[0], W.shape[2]), dtype=F8) for _ in range(2))
    used = torch.zeros(dC.shape[0], dtype=torch.bool)
    for e, a, b in spans(offsets):
        D[a:b] = dC[a:b] @ W[e]
        M[a:b] = dC[a:b].abs() @ W[e].abs()
        used[a:b] = True
    return D, M, used


def grouped_wgrad(dC, A, offsets, a_row):
    x, dC = gather(A, a_row, dC.shape[0]), d(dC)
    G = offsets.numel() - 1
    D, M = (torch.zeros((G, dC.shape[1], x.shape[1]), dtype=F8) for _ in range(2))
    for e, a, b in spans(offsets):
        D[e] = dC[a:b].T @ x[a:b]
        M[e] = dC[a:b].abs().T @ x[a:b].abs()
    return D, M


def combine(o, pos, w, add):
    o, pos = d(o), pos.cpu().long()
    T, k = pos.shape
    w = torch.ones((T, k), dtype=F8) if w is None else d(w)
    y = torch.zeros((T, o.shape[1]), dtype=F8) if add is None else d(add).clone()
    M = y.abs()
    for j in range(k):
        ok = ((pos[:, j] >= 0) & (pos[:, j] < o.shape[0]))[:, None]
        row = torch.where(ok, o[torch.where(ok[:, 0], pos[:, j], 0)], 0.0) if o.shape[0] else torch.zeros_like(y)
        y = y + w[:, j, None] * row
        M = M + (w[:, j, None] * row).abs()
    return y, M


def adapter(x, A, B, scale, ids, base):
    """(y, bound of the fp32 sum before it is stored, h, bound of h)."""
    x, A, B = d(x), d(A), d(B)
    n, r, K = A.shape
    s = torch.ones(n, dtype=F8) if scale is None else d(scale)
    y = torch.zeros((x.shape[0], B.shape[1]), dtype=F8) if base is None else d(base).clone()
    slack = torch.zeros_like(y)
    h, hs = (torch.zeros((x.shape[0], r), dtype=F8) for _ in range(2))
    for t, e in enumerate(ids.cpu().tolist()):
        if not 0 <= e < n:
            continue
        h[t] = s[e] * (A[e] @ x[t])
        hs[t] = s[e].abs() * sums(K, A[e].abs() @ x[t].abs()) + U * h[t].abs()
        slack[t] = B[e].abs() @ hs[t] + sums(r, y[t].abs() + B[e].abs() @ h[t].abs())
        y[t] = y[t] + B[e] @ h[t]
    return y, slack, h, hs


def adapter_grad(dy, x, A, B, scale, ids, dx_base):
    """((dx, slack), (dA, slack), (dB, slack)): values and bounds of the fp32 sums."""
    dy, x, A, B = d(dy), d(x), d(A), d(B)
    n, r, K = A.shape
    N, T = B.shape[1], x.shape[0]
    s = torch.ones(n, dtype=F8) if scale is None else d(scale)
    dx = torch.zeros((T, K), dtype=F8) if dx_base is None else d(dx_base).clone()
    dxs = torch.zeros_like(dx)
    dA, dAs = (torch.zeros_like(A) for _ in range(2))
    dB, dBs = (torch.zeros_like(B) for _ in range(2))
    ids = ids.cpu()
    for e in range(n):
        rows = (ids == e).nonzero()[:, 0]
        xe, ye = x[rows], dy[rows]
        h = s[e] * xe @ A[e].T
        hs = s[e].abs() * sums(K, xe.abs() @ A[e].abs().T) + U * h.abs()
        g = s[e] * ye @ B[e]
        gs = s[e].abs() * sums(N, ye.abs() @ B[e].abs()) + U * g.abs()
        dxs[rows] = gs @ A[e].abs() + sums(r, dx[rows].abs() + g.abs() @ A[e].abs())
        dx[rows] += g @ A[e]
        dA[e], dAs[e] = g.T @ xe, gs.T @ xe.abs() + sums(len(rows), g.abs().T @ xe.abs())
        dB[e], dBs[e] = ye.T @ h, ye.abs().T @ hs + sums(len(rows), ye.abs().T @ h.abs())
    return (dx, dxs), (dA, dAs), (dB, dBs)
