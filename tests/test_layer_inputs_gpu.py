"""A layer's forward and backward passes through the library's calls, as they are used together: the
affinity pass on inputs made here against the oracle, and the gradients of a whole layer against
torch's in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hna():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import head_neuron_affinity_amd as m
    m.lib()
    return m


def dev(layer):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) and not k.startswith("group_of") else v)
            for k, v in layer.items()}


@pytest.mark.parametrize("config,T,tol,kind", [(0, 200, 1e-4, "max"), (1, 300, 1e-2, "fro")])
def test_affinity_pass_on_a_layer_run_here(hna, config, T, tol, kind):
    """Tolerances: those of the affinity pass's own parity tests, since both sides read the same a, g, u, r."""
    L = dev(synth.make_config_layer(config, T=T))
    T, H, d = L["a"].shape
    G, dt, hidden = max(L["group_of_head"].tolist()) + 1, L["a"].dtype, L["W_o"].shape[0]
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T, n, d, generator=gen, device="cuda").to(dt) for n in (H, G, G))
    x = torch.randn(T, hidden, generator=gen, device="cuda")
    rows = hna.attention_rows(T, torch.tensor([0, 90, T], dtype=torch.int32, device="cuda"))
    w_o, w_down = hna.quant_rows(L["W_o"].contiguous()), hna.quant_rows(L["W_down"].contiguous())
    grp = L["group_of_head"].tolist()
    got = hna.layer_inputs(x, q, k, v, w_o, L["gamma"], L["W_gate"], L["W_up"], rows, w_down, cap=30.0, group_of_head=grp)
    # the same bits as the calls one by one
    a, _ = hna.attention(q, k, v, rows, cap=30.0, group_of_head=grp)
    y = hna.quant_matmul(*hna.quant_rows(a.view(T, -1)), *w_o, dtype=dt)
    x_in, n, r, _ = hna.block_norm(x, y, L["gamma"])
    g, u, h = hna.gated_ffn(n, L["W_gate"], L["W_up"])
    for name, t in dict(a=a, x_in=x_in, n=n, r=r, g=g, u=u, h=h).items():
        assert torch.equal(got[name], t), name
    L.update({name: got[name] for name in ("a", "g", "u", "r", "x_in", "r_next")})
    assert L["r_next"].shape == (T,) and (L["r_next"] > 0).all()
    scores = hna.affinity_layer(L)
    ref = oracle.affinity_layer({name: (t.cpu() if isinstance(t, torch.Tensor) else t) for name, t in L.items()})
    for key in ("S_fo", "S_add", "S_down"):
        s, e = scores[key].double().cpu().numpy(), ref[key]
        err = np.abs(s - e).max() / np.abs(e).max() if kind == "max" else np.linalg.norm(s - e) / np.linalg.norm(e)
        assert err <= tol, (key, err)


def test_gradients_of_a_whole_layer(hna):
    """x -> q, k, v -> attention -> W_o -> norm step -> gated FFN -> W_down, in fp32, each step's gradient
    by the library's call where it has one.  fp32 rounding is 6e-8 a step; a dozen products of up to 200 terms
    of either sign stay within 2e-5 of the gradients' norms."""
    T, C, H, G, d, I = 150, 64, 4, 2, 32, 200
    gen = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, gamma = r(T, C), 1 + 0.1 * r(C)
    w = {n: r(o, i) / i ** 0.5 for n, o, i in (("q", H * d, C), ("k", G * d, C), ("v", G * d, C), ("o", C, H * d), ("gate", I, C), ("up", I, C), ("down", C, I))}
    dout, rows = r(T, C), hna.attention_rows(T, torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda"))

    q, k, v = (x @ w[n].t() for n in "qkv")
    qh, kh, vh = q.view(T, H, d), k.view(T, G, d), v.view(T, G, d)
    a, lse = hna.attention(qh, kh, vh, rows, cap=10.0)
    x_in, n, rms, _ = hna.block_norm(x, a.view(T, -1) @ w["o"].t(), gamma)
    g, u, h = hna.gated_ffn(n, w["gate"], w["up"])
    # loss = sum((x_in + h W_down^T) dout)
    got = {"down": dout.t() @ h}
    dn, got["gate"], got["up"] = hna.gated_ffn_backward(dout @ w["down"], n, w["gate"], w["up"], g, u)
    back = hna.block_norm_backward(x_in, rms, dn=dn, dx_out=dout, gamma=gamma, want_dy=True)
    got["gamma"] = back["dgamma"]
    got["o"] = back["dy"].t() @ a.view(T, -1)
    da = (back["dy"] @ w["o"]).view(T, H, d)
    grads = hna.attention_backward(da, qh, kh, vh, a, lse, rows, cap=10.0)
    got["x"] = back["dx"]
    for name, t in zip("qkv", grads):
        t = t.reshape(T, -1)
        got[name] = t.t() @ x
        got["x"] = got["x"] + t @ w[name]

    wide = {name: t.double().requires_grad_(True) for name, t in dict(w, x=x, gamma=gamma).items()}
    X = wide["x"]
    Q, K, V = ((X @ wide[n].t()).view(T, -1, d) for n in "qkv")
    at = torch.arange(T, device="cuda")
    seen = (at[None] >= rows[:, :1]) & (at[None] < rows[:, 1:2])
    heads = []
    for i in range(H):
        s = 10 * torch.tanh(Q[:, i] @ K[:, i * G // H].t() * d ** -0.5 / 10)
        heads.append(torch.softmax(s.masked_fill(~seen, -torch.inf), 1) @ V[:, i * G // H])
    xi = X + torch.cat(heads, 1) @ wide["o"].t()
    nn = xi * torch.rsqrt(xi.square().mean(1, keepdim=True) + 1e-6) * wide["gamma"]
    out = xi + (torch.nn.functional.silu(nn @ wide["gate"].t()) * (nn @ wide["up"].t())) @ wide["down"].t()
    want = torch.autograd.grad((out * dout.double()).sum(), list(wide.values()))
    for name, e in zip(wide, want):
        assert (got[name].double() - e).norm() <= 2e-5 * e.norm(), name
