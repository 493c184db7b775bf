"""The gated FFN and its gradients against the formulas in 64 bits.

Tolerances count roundings.  A sum of K products in fp32 is off by at most about K 2^-24 of the sum of
their magnitudes, in any order; the result is then rounded to its type (half a step, eps / 2).  dg and du
are rounded to the type before the products that read them (eps / 2 of each), so a gradient is off by at
most eps / 2 of the sum of its terms' magnitudes more.  silu takes a few fp32 roundings (8 2^-24)."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def hna():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import head_neuron_affinity_amd as m
    m.lib()
    return m


def layer(T, C, I, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return r(T, C).to(dtype), (r(I, C) / C ** 0.5).to(dtype), (r(I, C) / C ** 0.5).to(dtype), r(T, I).to(dtype)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, want, slack, name):
    """|got - want| <= slack, elementwise, all in 64 bits; the worst element is named."""
    off = (got.double() - want).abs() - slack
    worst = off.max().item() if off.numel() else 0.0
    assert not torch.isnan(got).any() and worst <= 0, f"{name}: {worst:.3e} over its bound"


def check_forward(n, wg, wu, g, u, h, dtype):
    C = n.shape[1]
    nd, sums, exact = n.double(), {}, {}
    for k, w in (("g", wg), ("u", wu)):
        exact[k] = nd @ w.double().t()
        sums[k] = C * 2.0 ** -24 * (nd.abs() @ w.double().abs().t()) + 1e-30
    for k, t in (("g", g), ("u", u)):
        if t is not None:
            within(t, exact[k], sums[k] + half(dtype) * (exact[k].abs() + sums[k]), k)
    if h is not None:
        eg, eu = exact["g"], exact["u"]
        silu = eg * torch.sigmoid(eg)
        # |silu'| < 1.1; the sums' errors, then silu's own
        off = 1.1 * sums["g"] * (eu.abs() + sums["u"]) + silu.abs() * sums["u"] + 8 * 2.0 ** -24 * (1 + eg.abs()) * (silu * eu).abs()
        within(h, silu * eu, off + half(dtype) * ((silu * eu).abs() + off) + 1e-30, "h")


SIZES = [(1, 8, 1), (1, 4096, 333), (2, 64, 37), (5, 1024, 100), (16, 256, 2531), (33, 1000, 129), (64, 264, 64),
         (100, 72, 31), (219, 1000, 2531), (300, 520, 4096), (777, 1536, 130), (4100, 128, 2600), (2500, 1000, 4091)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,I", SIZES)
def test_forward(hna, T, C, I, dtype):
    n, wg, wu, _ = layer(T, C, I, dtype)
    g, u, h = hna.gated_ffn(n, wg, wu)
    check_forward(n, wg, wu, g, u, h, dtype)
    # each choice of outputs gives the same values
    for gu, hh in ((True, False), (False, True)):
        g2, u2, h2 = hna.gated_ffn(n, wg, wu, want_gu=gu, want_h=hh)
        assert (g2 is None, u2 is None, h2 is None) == (not gu, not gu, not hh)
        for a, b in ((g, g2), (u, u2), (h, h2)):
            assert b is None or torch.equal(a, b)


def exact_backward(dh, n, wg, wu, g, u):
    d, gd, ud = dh.double(), g.double(), u.double()
    sg = torch.sigmoid(gd)
    return d * ud * sg * (1 + gd * (1 - sg)), d * gd * sg


def check_backward(dh, n, wg, wu, g, u, dn, dwg, dwu, dtype):
    T, I = dh.shape
    dg, du = exact_backward(dh, n, wg, wu, g, u)
    # dg, du: a few fp32 roundings, exp's grow with |g|; then the type's
    gd, ud, d = g.double(), u.double(), dh.double()
    sg = torch.sigmoid(gd)
    loose = 8 * 2.0 ** -24 * (1 + gd.abs()) * sg
    og = (d * ud).abs() * loose * (1 + gd.abs()) + half(dtype) * dg.abs() + 1e-37
    ou = (d * gd).abs() * loose + half(dtype) * du.abs() + 1e-37
    W, N = [w.double() for w in (wg, wu)], n.double()
    if dn is not None:
        want = dg @ W[0] + du @ W[1]
        size = dg.abs() @ W[0].abs() + du.abs() @ W[1].abs()
        off = og @ W[0].abs() + ou @ W[1].abs() + (2 * I + 16) * 2.0 ** -24 * size
        within(dn, want, off + half(dtype) * (want.abs() + off) + 1e-30, "dn")
    for name, t, x, o in (("dw_gate", dwg, dg, og), ("dw_up", dwu, du, ou)):
        if t is not None:
            want = x.t() @ N
            off = o.t() @ N.abs() + T * 2.0 ** -24 * (x.abs().t() @ N.abs())
            within(t, want, off + half(dtype) * (want.abs() + off) + 1e-30, name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,C,I", SIZES)
def test_backward(hna, T, C, I, dtype):
    n, wg, wu, dh = layer(T, C, I, dtype, seed=1)
    g, u, _ = hna.gated_ffn(n, wg, wu, want_h=False)
    dn, dwg, dwu = hna.gated_ffn_backward(dh, n, wg, wu, g, u)
    check_backward(dh, n, wg, wu, g, u, dn, dwg, dwu, dtype)
    only = hna.gated_ffn_backward(dh, n, wg, wu, g, u, want_dw=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dn)
    only = hna.gated_ffn_backward(dh, n, wg, wu, g, u, want_dn=False)
    assert only[0] is None and torch.equal(only[1], dwg) and torch.equal(only[2], dwu)


def test_backward_against_differences(hna):
    """fp32: the loss sum(h dh) moves along a direction as the gradients say; central differences of
    step s are off by s^2 and by rounding / s."""
    n, wg, wu, dh = layer(40, 64, 72, F32, seed=2)
    g, u, _ = hna.gated_ffn(n, wg, wu)
    grads = hna.gated_ffn_backward(dh, n, wg, wu, g, u)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for x, grad in zip((n, wg, wu), grads):
        way = torch.randn(x.shape, generator=gen, device="cuda")
        way /= way.norm()
        loss = []
        for s in (1e-2, -1e-2):
            moved = [t + s * way if t is x else t for t in (n, wg, wu)]
            loss.append((hna.gated_ffn(*moved, want_gu=False)[2].double() * dh.double()).sum().item())
        along = (grad.double() * way.double()).sum().item()
        # |loss| is about sqrt(40 * 72) = 54 with sums of 64 products: its rounding is at most
        # 64 2^-24 of the terms' sum (40 * 72 * 1), 0.011, over 2e-2; in practice far less
        assert abs((loss[0] - loss[1]) / 2e-2 - along) <= 0.6, (loss, along)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_tokens(hna, dtype):
    n, wg, wu, dh = layer(0, 64, 33, dtype)
    g, u, h = hna.gated_ffn(n, wg, wu)
    assert g.shape == u.shape == h.shape == (0, 33)
    nan = torch.full_like(wg, float("nan"))
    dn, dwg, dwu = hna.gated_ffn_backward(dh, n, wg, wu, g, u, dw_gate=nan, dw_up=nan.clone())
    assert dn.shape == (0, 64) and not dwg.any() and not dwu.any()


@pytest.mark.parametrize("T,C,I", [(7, 64, 37), (300, 264, 130), (2600, 128, 4100)])
def test_bad_rows_stay_alone(hna, T, C, I):
    n, wg, wu, dh = layer(T, C, I, BF16, seed=3)
    clean = hna.gated_ffn(n, wg, wu)
    dn = hna.gated_ffn_backward(dh, n, wg, wu, *clean[:2], want_dw=False)[0]
    bad = [0, T // 2, T - 1]
    n2, dh2 = n.clone(), dh.clone()
    n2[bad[0]], n2[bad[1]], n2[bad[2]] = float("nan"), float("inf"), float("-inf")
    dh2[bad] = float("nan")
    good = torch.tensor([t not in bad for t in range(T)], device="cuda")
    for a, b in zip(clean, hna.gated_ffn(n2, wg, wu)):
        assert torch.equal(a[good], b[good]) and not torch.isfinite(b[~good]).all()
    got = hna.gated_ffn_backward(dh2, n, wg, wu, *clean[:2], want_dw=False)[0]
    assert torch.equal(got[good], dn[good]) and torch.isnan(got[~good]).all()


def test_rows_behind_are_left(hna):
    n, wg, wu, _ = layer(50, 64, 37, BF16)
    whole = [torch.full((60, 37), 7.0, dtype=BF16, device="cuda") for _ in range(3)]
    hna.gated_ffn(n, wg, wu, g=whole[0][:50], u=whole[1][:50], h=whole[2][:50])
    assert all((w[50:] == 7).all() for w in whole)


def test_repeats_and_streams(hna):
    """Two streams at once, each with its own outputs and workspace; every repeat gives the same bits."""
    made = [layer(T, 256, 515, BF16, seed=T) for T in (130, 700)]
    want = []
    for n, wg, wu, dh in made:
        g, u, h = hna.gated_ffn(n, wg, wu)
        want.append((g, u, h, *hna.gated_ffn_backward(dh, n, wg, wu, g, u)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = []
    for _ in range(3):
        for s, (n, wg, wu, dh) in zip(streams, made):
            with torch.cuda.stream(s):
                g, u, h = hna.gated_ffn(n, wg, wu)
                got.append((g, u, h, *hna.gated_ffn_backward(dh, n, wg, wu, g, u)))
    torch.cuda.synchronize()
    for x, y in zip(itertools.cycle(want), got):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_captured(hna):
    n, wg, wu, dh = layer(200, 128, 300, BF16, seed=9)
    dims = hna.hna_ffn_dims(200, 128, 300, hna.HNA_BF16)
    ws = torch.empty(hna.gated_ffn_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    out = [torch.empty(200, 300, dtype=BF16, device="cuda") for _ in range(3)]
    grads = [torch.empty_like(t) for t in (n, wg, wu)]

    def step():
        hna.gated_ffn(n, wg, wu, g=out[0], u=out[1], h=out[2])
        hna.gated_ffn_backward(dh, n, wg, wu, out[0], out[1], dn=grads[0], dw_gate=grads[1], dw_up=grads[2], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        n.copy_(torch.randn(200, 128, device="cuda"))
        for t in (*out, *grads):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (*out, *grads)]
        g, u, h = hna.gated_ffn(n, wg, wu)
        eager = (g, u, h, *hna.gated_ffn_backward(dh, n, wg, wu, g, u))
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), k
