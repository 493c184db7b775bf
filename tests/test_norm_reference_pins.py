"""The 64-bit reference of the norm step's gradients against central differences and automatic
differentiation of its forward formula (CPU)."""
import pytest
import torch

import norm_reference as ref


def made(T, C, gate_tokens, post, seed=3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(x=n(T, C), y=n(T, C), gamma=1 + 0.1 * n(C), gamma_post=1 + 0.1 * n(C) if post else None,
                gate=n(-(-T // gate_tokens), C) if gate_tokens else None), n(T, C), n(T, C)


@pytest.mark.parametrize("gate_tokens", [0, 1, 2, 5])
@pytest.mark.parametrize("post", [False, True])
def test_gradients_against_differences_and_autograd(gate_tokens, post):
    T, C = 5, 16
    a, dn, dx_out = made(T, C, gate_tokens, post)
    step = dict(res_scale=0.75, block_scale=1.5)

    def loss(**t):
        h, _, _ = ref.join(t["x"], t["y"], t["gamma_post"], t["gate"], gate_tokens or None, eps=1e-6, **step)
        n, _ = ref.norm(h, t["gamma"], 1e-6)
        return (n * dn).sum() + (h * dx_out).sum()

    h, _, r_post = ref.join(a["x"], a["y"], a["gamma_post"], a["gate"], gate_tokens or None, eps=1e-6, **step)
    _, r = ref.norm(h, a["gamma"], 1e-6)
    got = ref.gradients(h, r, dn, dx_out, a["gamma"], a["y"], a["gamma_post"], r_post, a["gate"],
                        gate_tokens or None, **step)
    leaves = {k: v.clone().requires_grad_() for k, v in a.items() if v is not None}
    loss(**{**a, **leaves}).backward()
    for k, leaf in leaves.items():
        g = got["d" + k][0]
        assert torch.allclose(g, leaf.grad, rtol=1e-10, atol=1e-12), k
        v = torch.randn(leaf.shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
        e = 1e-5
        diff = (loss(**{**a, k: a[k] + e * v}) - loss(**{**a, k: a[k] - e * v})) / (2 * e)
        assert abs(float((g * v).sum() - diff)) <= 1e-7 * (1 + abs(float(diff))), k


def test_quant_reference_ties_go_to_even():
    x = torch.tensor([[254.0, 1.0, 3.0, -1.0, -3.0, 127.0, 0.0]], dtype=torch.float64)   # 0.5, 1.5, .., 63.5
    q, s = ref.quant(x)
    assert q.tolist() == [[127.0, 0.0, 2.0, 0.0, -2.0, 64.0, 0.0]] and s.item() == 2.0
