"""The norm step, its gradients and 8-bit rows in 64 bits, from their formulas, with error bounds.

Each `*_bound` says how far a result held in fp32 and rounded once to its type may be off: half a
step of its type, and a count of fp32 roundings (2^-24 each) times the magnitudes that enter.  A sum
over a row runs over at most 16 terms in a lane, 6 steps across a wave and 15 across waves; with the
mean, eps, the root and the products around it no value collects more than ROUNDINGS of them.
"""
import torch

ROUNDINGS = 64
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gate_rows(gate, gate_tokens, T):
    return gate[torch.arange(T, device=gate.device) // gate_tokens]


def join(x, y=None, gamma_post=None, gate=None, gate_tokens=None, res_scale=1.0, block_scale=1.0, eps=1e-6):
    """(x' unrounded, the block's part of it, r_post or None); all arguments in 64 bits."""
    if y is None:
        return x, torch.zeros_like(x), None
    r_post = None
    b = y
    if gamma_post is not None:
        r_post = torch.sqrt((y * y).mean(1) + eps)
        b = torch.where(r_post[:, None] > 0, y / r_post[:, None], 0.0) * gamma_post
    if gate is not None:
        b = b * gate_rows(gate, gate_tokens, x.shape[0])
    return res_scale * x + block_scale * b, block_scale * b, r_post


def norm(h, gamma=None, eps=1e-6):
    """(n, r) of rows h in 64 bits."""
    r = torch.sqrt((h * h).mean(1) + eps)
    n = torch.where(r[:, None] > 0, h / r[:, None], 0.0)
    return (n if gamma is None else n * gamma), r


def quant(x):
    """(q, scale) of rows in 64 bits: the quotient of a value that lies on a half is exact."""
    top = x.abs().amax(1)
    q = torch.where(top[:, None] > 0, torch.round(127.0 * x / top[:, None]), 0.0)
    return q, top / 127.0


def gradients(h, r, dn=None, dx_out=None, gamma=None, y=None, gamma_post=None, r_post=None, gate=None,
              gate_tokens=None, res_scale=1.0, block_scale=1.0):
    """{name: (value, magnitude of the terms it is made of)}; all arguments in 64 bits."""
    T, C = h.shape
    d = torch.zeros_like(h)
    m = torch.zeros_like(h)
    out = {}
    if dx_out is not None:
        d, m = dx_out, dx_out.abs()
    if dn is not None:
        inv = torch.where(r > 0, 1 / r, 0.0)[:, None]
        xh = h * inv
        w = dn if gamma is None else dn * gamma
        d = d + (w - xh * (w * xh).mean(1, keepdim=True)) * inv
        m = m + (w.abs() + xh.abs() * (w * xh).abs().mean(1, keepdim=True)) * inv
        out["dgamma"] = ((dn * xh).sum(0), (dn * xh).abs().sum(0))
    out["dx"] = (res_scale * d, abs(res_scale) * m)
    d, m = block_scale * d, abs(block_scale) * m
    g = torch.ones_like(h) if gate is None else gate_rows(gate, gate_tokens, T)
    if y is not None:
        inv = torch.ones(T, 1, dtype=h.dtype, device=h.device)
        if gamma_post is not None:
            inv = torch.where(r_post > 0, 1 / r_post, 0.0)[:, None]
        gp = torch.ones(C, dtype=h.dtype, device=h.device) if gamma_post is None else gamma_post
        yh = y * inv
        if gate is not None:
            rows = torch.arange(T, device=h.device) // gate_tokens
            zero = torch.zeros_like(gate)
            out["dgate"] = (zero.index_add(0, rows, d * yh * gp), zero.index_add(0, rows, m * (yh * gp).abs()))
    d, m = d * g, m * g.abs()
    if gamma_post is not None:
        out["dgamma_post"] = ((d * yh).sum(0), (m * yh.abs()).sum(0))
        v, mv = d * gp, m * gp.abs()
        d = (v - yh * (v * yh).mean(1, keepdim=True)) * inv
        m = (mv + yh.abs() * (mv * yh.abs()).mean(1, keepdim=True)) * inv
    out["dy"] = (d, m)
    return out


def assert_within(got, want, magnitude, dtype, what, roundings=ROUNDINGS):
    """|got - want| <= half a step of want + `roundings` fp32 roundings of `magnitude` (and fp32's
    smallest normal, for values below it)."""
    want = want.to(got.device)
    bound = half_step(dtype) * want.abs() * (1 + 1e-3) + roundings * U * magnitude.to(got.device) + 1.2e-38
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off by more than their bound, "
        f"worst {float((off / bound).nan_to_num(9e9).max()):.3g} times it")
