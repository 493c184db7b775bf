"""Attention, its gradients and single tokens in 64 bits from the formulas, with what fp32 sums and
roundings to the inputs' type may take from each result.

A sum of n products in fp32 is off by at most about n 2^-24 of the sum of their magnitudes.  A score's
error e moves its exponential by e of its value.  exp(s - m), p and ds are rounded to the inputs' type (half
a step, eps / 2) before they meet v, da, k and q; results are rounded once more."""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def seen_by(T, rows, causal=True, device="cuda"):
    """[T, T]: query i sees key j; and [T]: the token is of a document."""
    j = torch.arange(T, device=device)
    if rows is None:
        lo, hi = torch.zeros_like(j), (j + 1 if causal else torch.full_like(j, T))
        return (j[None] >= lo[:, None]) & (j[None] < hi[:, None]), torch.ones(T, dtype=torch.bool, device=device)
    lo, hi = rows[:, 0].long(), rows[:, 1].long()
    return (j[None] >= lo[:, None].clamp_min(0)) & (j[None] < hi[:, None]) & (lo >= 0)[:, None], lo >= 0


def scores(q, k, at, scale, cap, slope):
    """One head's scores [n, m] in 64 bits, 1 - tanh^2, and a bound on the error that fp32 brings."""
    q, k = q.double(), k.double()
    raw = scale * (q @ k.t())
    off = U * scale * (q.shape[1] + 8) * (q.abs() @ k.abs().t())
    bent = torch.ones_like(raw)
    s = raw
    if cap > 0:
        t = torch.tanh(raw / cap)
        s, bent, off = cap * t, 1 - t * t, off + 8 * U * cap
    if slope is not None:
        far = (torch.arange(k.shape[0], device=q.device)[None] - at[:, None]).abs().double()
        s = s - slope.double() * far
        off = off + 8 * U * (slope.double() * far).abs()
    return s, bent, off + 4 * U * s.abs()


def softmax(s, seen):
    """Weights and lse of the seen scores; rows that see nothing have weights 0 and lse -inf."""
    z = torch.where(seen, s, -torch.inf)
    lse = torch.logsumexp(z, 1)
    return torch.where(seen, torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)[:, None]), 0.0), lse


def groups(H, G, group_of_head):
    return [h * G // H for h in range(H)] if group_of_head is None else list(group_of_head)


def forward(q, k, v, seen, scale, cap, slopes, group_of_head):
    """(a, lse) and their bounds, 64 bits."""
    T, H, d = q.shape
    at = torch.arange(T, device=q.device)
    a, lse, off_a, off_l = (torch.zeros(*sh, dtype=torch.float64, device=q.device) for sh in ((T, H, d), (T, H), (T, H, d), (T, H)))
    for h, g in enumerate(groups(H, k.shape[1], group_of_head)):
        s, _, e = scores(q[:, h], k[:, g], at, scale, cap, None if slopes is None else slopes[h])
        w, lse[:, h] = softmax(s, seen)
        e = torch.where(seen, e, 0.0).amax(1, keepdim=True) + (k.shape[0] + 16) * U + U * s.abs().amax(1, keepdim=True)
        vd = v[:, g].double()
        a[:, h] = w @ vd
        off_a[:, h] = (half(q.dtype) + 2 * e) * (w @ vd.abs()) + half(q.dtype) * a[:, h].abs()
        off_l[:, h] = (e[:, 0] + 8 * U * lse[:, h].abs().nan_to_num(0, 0, 0))
    return a, lse, off_a + 1e-30, off_l + 1e-30


def backward(da, q, k, v, a, lse, seen, scale, cap, slopes, group_of_head):
    """{name: (gradient, bound)} from the a and lse that are given, 64 bits."""
    T, H, d = q.shape
    G = k.shape[1]
    at = torch.arange(T, device=q.device)
    hf = half(q.dtype)
    z = lambda heads: torch.zeros(T, heads, d, dtype=torch.float64, device=q.device)  # noqa: E731
    got = {n: (z(x), z(x)) for n, x in (("dq", H), ("dk", G), ("dv", G))}

    def add(name, h, left, err, right):
        """left @ right, left's error err, fp32 sums"""
        x, o = got[name]
        x[:, h] += left @ right
        o[:, h] += err @ right.abs() + (right.shape[0] + 16) * U * (left.abs() @ right.abs())

    for h, g in enumerate(groups(H, G, group_of_head)):
        s, bent, e = scores(q[:, h], k[:, g], at, scale, cap, None if slopes is None else slopes[h])
        ls = lse[:, h].double()[:, None]
        on = seen & torch.isfinite(ls)
        p = torch.where(on, torch.exp(torch.where(on, s - ls, 0.0)), 0.0)
        rel = e + 4 * U * ls.abs().nan_to_num(0, 0, 0) + 16 * U
        A, V, dA = a[:, h].double(), v[:, g].double(), da[:, h].double()
        dp, D = dA @ V.t(), (dA * A).sum(1, keepdim=True)
        ds = p * (dp - D) * bent
        off = p * ((d + 8) * U * (dA.abs() @ V.abs().t() + (dA * A).abs().sum(1, keepdim=True)) + rel * (dp - D).abs() * bent + 8 * U * (dp - D).abs())
        Q, K = q[:, h].double(), k[:, g].double()
        add("dv", g, p.t(), (p * (rel + hf)).t(), dA)
        add("dq", h, ds * scale, (off + hf * ds.abs()) * scale, K)
        add("dk", g, ds.t() * scale, (off + hf * ds.abs()).t() * scale, Q)
    return {n: (x, o + hf * (x.abs() + o) + 1e-30) for n, (x, o) in got.items()}
