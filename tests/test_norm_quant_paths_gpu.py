"""Paths of the norm step and the 8-bit calls that ordinary sizes do not reach: values that one output
must not read, layers of either type, large calls, and calls behind work on another stream."""
import numpy as np
import pytest
import torch

import norm_reference as ref
import oracle
import synth
from test_norm_quant_gpu import BF, F, NAN, Step, check_product, gen, hna, int_rows, wide  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- gradients and y
@pytest.mark.parametrize("C", [72, 1496, 4096])
@pytest.mark.parametrize("gate", [1, 4, 12])
@pytest.mark.parametrize("with_dn", [False, True])
def test_backward_dy_without_block_norm_does_not_read_y(hna, C, gate, with_dn):
    """Without a block norm dy = block_scale gate d: an infinity or a NaN in y reaches dgate's element of
    that column and gate row only.  At the x' of a clean forward call; dx, dy and dgamma as with clean y,
    bit for bit."""
    s = Step(12, C, F, BF, post=False, gate=gate)
    x_out, _, r, _ = s.forward(hna.block_norm)
    kw = {} if with_dn else dict(dn=None)
    clean = s.backward(hna, x_out, r, None, **kw)
    s.check_backward(clean, x_out, r, None, dn=with_dn)
    y = s.y.clone()
    bad = [(0, 3), (5, 0), (11, C - 1)]
    for (t, c), v in zip(bad, (float("inf"), NAN, -float("inf"))):
        y[t, c] = v
    got = s.backward(hna, x_out, r, None, y=y, **kw)
    for k in ("dx", "dy", "dgamma"):
        same = got[k] is None or torch.equal(got[k], clean[k])
        assert same, k
    hit = torch.zeros(s.gate.shape, dtype=torch.bool, device="cuda")
    for t, c in bad:
        hit[t // gate, c] = True
    same = torch.equal(got["dgate"][~hit], clean["dgate"][~hit])
    assert same and not bool(torch.isfinite(got["dgate"][hit]).any())


# ---------------------------------------------------------------- layers of either type
@pytest.mark.parametrize("config,T", [(0, 256), (1, 130)])
def test_layer_inputs_in_the_layers_own_type(hna, config, T):
    """layer.update(FfnInputs(layer).run(layer["x_in"])), then the affinity pass and the leave-one-out
    score, on an fp32 and a bf16 layer: g and u in the layer's type, the scores against the oracle on
    the same r, g and u."""
    L = synth.make_config_layer(config, T=T, with_x=True)
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) and not k.startswith("group_of") else v) for k, v in L.items()}
    fp32 = L["a"].dtype == F
    g, u, r = dev["g"], dev["u"], dev["r"]
    dev.update(hna.FfnInputs(dev, eps=0.0).run(dev["x_in"]))
    assert dev["g"].dtype == dev["u"].dtype == L["a"].dtype and dev["x_in"].dtype == F
    ref.assert_within(dev["r"], r.double(), r.double(), F, "r")
    for k, want in (("g", g), ("u", u)):
        # a uniform error of one step of max / 127 is max / 440 rms; max <= 5 rms: W and n bring 1.2% each
        rel = float((dev[k].double() - want.double()).norm() / want.double().norm())
        assert rel < 0.024, (k, rel)
    ap = hna.pass_for_layer(dev)
    got = ap.run(dev)
    loo = ap.loo(dev, [int(x) for x in dev["group_of_head"].tolist()])
    torch.cuda.synchronize()
    want = oracle.affinity_layer({**L, **{k: dev[k].cpu() for k in ("r", "g", "u")}})

    def check(x, w, what):
        x, w = x.double().cpu().numpy(), np.asarray(w)
        if fp32:
            assert np.max(np.abs(x - w)) <= 1e-4 * np.max(np.abs(w)), what
        else:
            assert np.linalg.norm(x - w) <= 1e-2 * np.linalg.norm(w), what

    for k in ("S_fo", "S_add", "S_down"):
        check(got[k], want[k], k)
    assert loo.shape == got["S_fo"].shape and bool(torch.isfinite(loo).all())


def test_layer_inputs_take_a_type(hna):
    """ffn_inputs with each type of g and u: the same sums and scales, rounded once or not."""
    s = Step(33, 520, F, BF)
    w = [hna.quant_rows(torch.randn(200, 520, generator=torch.Generator().manual_seed(k)).cuda()) for k in (1, 2)]
    kw = dict(y=s.y, gamma_post=s.gamma_post, res_scale=s.rs, block_scale=s.bs, eps=s.eps)
    wide_out = hna.ffn_inputs(s.x, s.gamma, *w, dtype=F, **kw)
    short = hna.ffn_inputs(s.x, s.gamma, *w, **kw)
    for k in ("g", "u"):
        assert wide_out[k].dtype == F and short[k].dtype == BF
        same = torch.equal(wide_out[k].bfloat16(), short[k])
        assert same, k
    with pytest.raises(TypeError):
        hna.ffn_inputs(s.x, s.gamma, *w, dtype=torch.float16, **kw)


# ------------------------------------------------------------------------- large calls
# widths of every lane count a row is spread over: 64 lanes (8 and 16 elements each), 128, .. 1024
WIDTHS = [504, 1000, 2040, 4088, 8184, 16376]
PAST_CACHES = 256 << 20                            # calls that move more go past the caches, on another grid


def lanes(C):
    return 64 if C <= 1024 else 128 if C <= 2048 else 256 if C <= 4096 else 512 if C <= 8192 else 1024


def check_step(hna, s):
    """Forward, 8-bit forward and backward (with and without y) of one large step against 64 bits, again in
    place bit for bit."""
    x_out, n, r, r_post = s.forward(hna.block_norm)
    want = s.check_join(x_out, r, r_post)
    ref.assert_within(n, want, want.abs(), s.io, "n")
    xq, q, scale, rq, rpq = s.forward(hna.block_norm_quant)
    same = [torch.equal(a, b) for a, b in ((xq, x_out), (rq, r), (rpq, r_post))]
    assert all(same), same
    top = want.abs().amax(1)
    ref.assert_within(scale, top / 127, top / 127, F, "scale")
    want.mul_((127 / top)[:, None])
    off = float((q[:, :s.C].double() - want).abs().max())   # as in test_norm_quant
    assert off <= 0.501 and not bool(q[:, s.C:].any()), off
    del xq, q, want
    # terms with ROUNDINGS each, then additions: one lane's rows (a workgroup's T / n_wg over the rows it has
    # side by side), those rows' 4 sums, and the partial rows' 16 in a lane and a tree of 8
    side, wgs = max(1, 256 // lanes(s.C)), 512 if lanes(s.C) <= 256 else 256
    sums = ref.ROUNDINGS + -(-s.T // (side * wgs)) + side + 32
    for keep_y in (True, False):
        kw = {} if keep_y else dict(y=None, gamma_post=None)
        y, gp, rp = (s.y, s.gamma_post, r_post) if keep_y else (None, None, None)
        got = s.backward(hna, x_out, r, rp, **kw)
        w = ref.gradients(wide(x_out), wide(r), wide(s.dn), wide(s.dx_out), wide(s.gamma), wide(y), wide(gp), wide(rp),
                          wide(s.gate), s.gate_tokens, s.rs, s.bs)
        for k, dtype in (("dx", s.res), ("dy", s.io), ("dgamma", F), ("dgamma_post", F), ("dgate", s.io)):
            if k in w:
                ref.assert_within(got[k], *w.pop(k), dtype, k, sums if k.startswith("dg") else ref.ROUNDINGS)
        dn, dx_out = s.dn.clone(), s.dx_out.clone()
        again = s.backward(hna, x_out, r, rp, dn=dn, dx_out=dx_out, dx=dx_out, dy=dn, **kw)
        same = {k: got[k] is None or torch.equal(got[k], again[k]) for k in got}
        assert all(same.values()), same
    x, y = s.x, s.y
    s.x, s.y = x.clone(), y.clone()
    s.forward(hna.block_norm, x_out=s.x, n=s.y)
    same = torch.equal(s.x, x_out) and torch.equal(s.y, n)
    assert same


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("res,io", [(BF, BF), (F, BF), (F, F), (BF, F)])
def test_norm_calls_past_the_caches(hna, C, res, io):
    """Each of the four kinds of call moves more than 256 MB, on a number of rows that nothing divides."""
    size = lambda t: 2 if t == BF else 4  # noqa: E731
    T = PAST_CACHES // (C * (2 * size(res) + size(io) + 1)) + 7      # the 8-bit form moves least
    T += 1 - T % 2
    print(f"past the caches T={T} C={C} {res} {io}", flush=True)
    check_step(hna, Step(T, C, res, io, gate=T // 3))


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("res,io", [(BF, BF), (F, BF)])
def test_norm_calls_of_many_rows_a_workgroup(hna, C, res, io):
    """Below that size: every workgroup of a full grid (2048 lanes on each of 256 CUs) goes on to a second
    row, some to a third."""
    T = 256 * 2048 // lanes(C) * 2 + 3
    assert T * C * (12 if res == F else 8) < PAST_CACHES
    print(f"rows a workgroup T={T} C={C} {res} {io}", flush=True)
    check_step(hna, Step(T, C, res, io, gate=5))


@pytest.mark.parametrize("K", [504, 1000, 1528, 2040, 4088, 8184, 16376])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("large", [False, True])
def test_quant_rows_of_many_rows_a_workgroup(hna, K, dtype, large):
    """8-bit rows, exactly, where workgroups go on to further rows: within the caches and past them, and
    (K off 8) element by element."""
    for k in (K, K - 3):
        if large:
            rows = PAST_CACHES // (k * (2 if dtype == BF else 4) + k) + 7
        else:
            rows = 2 * 8192 + 3 if K <= 2048 else 3 * 2048 + 3 if K <= 8192 else 2 * 1024 + 3
            assert rows * k * 5 < PAST_CACHES
        print(f"8-bit rows {rows} x {k} {dtype}", flush=True)
        x = torch.randn(rows, k, generator=torch.Generator(device="cuda").manual_seed(k), device="cuda").to(dtype)
        x[rows - 2] = 0
        q, scale = hna.quant_rows(x)
        want, s = ref.quant(x.double())
        same = torch.equal(q[:, :k].double(), want) and not bool(q[:, k:].any())
        assert same
        ref.assert_within(scale, s, s, F, "scale", 0)


# ------------------------------------------------------- behind work on another stream
def behind_work(tensors, call):
    """`call` on a side stream whose queue is busy, with `tensors` holding other values until just before
    it on that stream: its outputs.  A launch or a copy made on another stream runs at once and reads the
    other values."""
    real = [t.clone() for t in tensors]
    big = torch.randn(4096, 4096, device="cuda")
    for t in tensors:
        t.fill_(NAN) if t.dtype.is_floating_point else t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(8):                         # some ms; the host is done with all below before that
            big = big @ big * 1e-3
        for t, v in zip(tensors, real):
            t.copy_(v)
        got = call()
        assert not side.query()
    torch.cuda.synchronize()
    return got


def streams_case(hna, name):
    """(inputs, call) of one entry point; call() returns its outputs."""
    s = Step(200, 1024, BF, BF, gate=50)
    if name in ("block_norm", "block_norm_quant"):
        return [s.x, s.y, s.gamma, s.gamma_post, s.gate], lambda: s.forward(getattr(hna, name))
    if name == "block_norm_backward":
        x_out, _, r, r_post = s.forward(hna.block_norm)
        return ([s.dn, s.dx_out, x_out, r, r_post, s.y, s.gamma, s.gamma_post, s.gate],
                lambda: tuple(s.backward(hna, x_out, r, r_post).values()))
    if name == "quant_rows":
        return [s.x], lambda: hna.quant_rows(s.x)
    w = [t for k in (1, 2) for t in hna.quant_rows(torch.randn(264, 1024, device="cuda"))]
    if name == "ffn_inputs":
        return ([s.x, s.y, s.gamma, *w],
                lambda: tuple(hna.ffn_inputs(s.x, s.gamma, w[:2], w[2:], y=s.y).values()))
    q, scale = hna.quant_rows(s.x)
    if name == "quant_matmul":
        return [q, scale, *w[:2]], lambda: (hna.quant_matmul(q, scale, *w[:2]),)
    return [q, scale, *w], lambda: hna.quant_matmul_pair(q, scale, *w)


@pytest.mark.parametrize("name", ["block_norm", "block_norm_quant", "block_norm_backward", "quant_rows", "quant_matmul",
                                  "quant_matmul_pair", "ffn_inputs"])
def test_calls_run_in_their_streams_order(hna, name):
    tensors, call = streams_case(hna, name)
    want = call()
    torch.cuda.synchronize()
    got = behind_work(tensors, call)
    same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert len(same) == len(want) and all(same), same


# -------------------------------------------------------- few tokens, many channels
@pytest.mark.parametrize("T,N,K", [(1, 41000, 272), (4, 50003, 130), (2, 65536, 1024), (3, 12800, 4096), (5, 41000, 272)])
def test_product_of_few_tokens_with_many_channels(hna, T, N, K):
    print(f"few tokens T={T} N={N} K={K}", flush=True)
    g = gen(T + N + K)
    q, s = int_rows(g, T, K)
    w, ws = int_rows(g, N, K)
    for dtype in (BF, F):
        check_product(hna, q, s, w, ws, dtype)
    w1, s1 = int_rows(g, N // 2, K)
    for got, (m, c) in zip(hna.quant_matmul_pair(q, s, w[:N // 2], ws[:N // 2].clone(), w1, s1),
                           ((w[:N // 2], ws[:N // 2].clone()), (w1, s1))):
        same = torch.equal(got, hna.quant_matmul(q, s, m, c))
        assert same


@pytest.mark.parametrize("T,N,K", [(300, 2531, 1008), (300, 2531, 1024), (190, 4096, 1030), (64, 12290, 2048), (20, 14336, 1500)])
def test_product_of_one_round_of_tiles(hna, T, N, K):
    """128 to 256 tiles of 64 x 64, k at both sides of the border between its two forms."""
    print(f"one round T={T} N={N} K={K}", flush=True)
    g = gen(T + N + K)
    q, s = int_rows(g, T, K)
    w, ws = int_rows(g, N, K)
    for dtype in (BF, F):
        check_product(hna, q, s, w, ws, dtype)


# ------------------------------------------------------------ rows past fp32's squares
@pytest.mark.parametrize("C", [520, 4096])
def test_rows_whose_squares_pass_fp32(hna, C):
    """Finite values whose sum of squares is none: r = inf and n = 0, as the header says, x' right, the rows
    beside it as without it."""
    s = Step(5, C, F, F, post=False)
    clean = s.forward(hna.block_norm)
    s.x[2, 7] = 1e25
    x_out, n, r, _ = s.forward(hna.block_norm)
    _, q, scale, _, _ = s.forward(hna.block_norm_quant)
    assert float(r[2]) == float("inf") and not bool(n[2].any()) and not bool(q[2].any()) and float(scale[2]) == 0
    want = s.rs * float(s.x[2, 7])                 # lies halfway between two fp32 values: either is right
    assert abs(float(x_out[2, 7]) - want) <= 2.0 ** -24 * want
    others = [0, 1, 3, 4]
    same = [torch.equal(a[others], b[others]) for a, b in zip((x_out, n, r), clean)]
    assert all(same), same
