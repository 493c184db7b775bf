"""The norm step between blocks, its gradients, 8-bit rows and their product against the 64-bit
reference (norm_reference.py), whose bounds were derived from the formulas and the count of roundings."""
import pytest
import torch

import norm_reference as ref
import oracle
import synth

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def hna():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import head_neuron_affinity_amd as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def wide(t):
    return None if t is None else t.double()


class Step:
    """Arguments of one norm step; `gate`: tokens per gate row, 0 for none."""

    def __init__(self, T, C, res, io, y=True, post=True, gate=0, gamma=True, rs=0.75, bs=1.5, eps=1e-6, seed=1):
        g = gen(seed * 7919 + T * 31 + C)
        self.T, self.C, self.eps, self.gate_tokens = T, C, eps, gate or None
        self.x = randn(g, T, C, dtype=res, scale=2.0)
        self.y = randn(g, T, C, dtype=io, scale=0.7) if y else None
        self.gamma = 1 + 0.2 * randn(g, C) if gamma else None
        self.gamma_post = 1 + 0.2 * randn(g, C) if y and post else None
        self.gate = randn(g, -(-T // gate), C, dtype=io) if gate and T else None
        if self.gate is None:
            self.gate_tokens = None
        self.rs, self.bs = (rs, bs) if y else (1.0, 1.0)
        self.io, self.res = io if y else res, res
        self.dn = randn(g, T, C, dtype=self.io)
        self.dx_out = randn(g, T, C, dtype=res)

    def forward(self, call, **kw):
        return call(self.x, self.y, self.gamma, gamma_post=self.gamma_post, gate=self.gate,
                    gate_tokens=self.gate_tokens, res_scale=self.rs, block_scale=self.bs, eps=self.eps, **kw)

    def check_join(self, x_out, r, r_post):
        """x' and both r against 64 bits; returns x' as stored, in 64 bits."""
        if self.y is None:
            assert torch.equal(x_out, self.x)
        else:
            want, block, rp = ref.join(wide(self.x), wide(self.y), wide(self.gamma_post), wide(self.gate),
                                       self.gate_tokens, self.rs, self.bs, self.eps)
            ref.assert_within(x_out, want, block.abs() + want.abs(), self.res, "x_out")
            if rp is not None:
                ref.assert_within(r_post, rp, rp, F, "r_post")
        n, rr = ref.norm(wide(x_out), wide(self.gamma), self.eps)
        ref.assert_within(r, rr, rr, F, "r")
        return n

    def backward(self, hna, x_out, r, r_post, **kw):
        a = dict(dn=self.dn, dx_out=self.dx_out, gamma=self.gamma, y=self.y, gamma_post=self.gamma_post,
                 r_post=r_post, gate=self.gate, gate_tokens=self.gate_tokens, res_scale=self.rs,
                 block_scale=self.bs, want_dy=True)
        a.update(kw)
        return hna.block_norm_backward(x_out, r, **a)

    def check_backward(self, got, x_out, r, r_post, dn=True, dx_out=True):
        want = ref.gradients(wide(x_out), wide(r), wide(self.dn) if dn else None,
                             wide(self.dx_out) if dx_out else None, wide(self.gamma), wide(self.y),
                             wide(self.gamma_post), wide(r_post), wide(self.gate), self.gate_tokens,
                             self.rs, self.bs)
        for k, dtype in (("dx", self.res), ("dy", self.io), ("dgamma", F), ("dgamma_post", F), ("dgate", self.io)):
            if got[k] is None:
                assert k not in want or (k == "dgamma" and (self.gamma is None or not dn)), k
                continue
            assert got[k].dtype == dtype, k
            # sums over tokens: up to 64 more additions in a row of one lane's terms
            ref.assert_within(got[k], *want[k], dtype, k, 2 * ref.ROUNDINGS if k.startswith("dg") else ref.ROUNDINGS)


# ----------------------------------------------------------------------------- forward
SIZES = [(1, 8), (3, 64), (37, 520), (1, 1024), (130, 1000), (5, 1032), (2, 1536), (9, 2056), (4, 4096), (3, 8192),
         (2, 8200), (2, 16384), (700, 256)]
TYPES = [(BF, BF), (F, BF), (F, F), (BF, F)]


@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("res,io", TYPES)
def test_norm_step_sizes_and_types(hna, T, C, res, io):
    print(f"norm step T={T} C={C} {res} {io}", flush=True)
    for kw in (dict(), dict(y=False), dict(post=False, gate=3)):
        s = Step(T, C, res, io, **kw)
        x_out, n, r, r_post = s.forward(hna.block_norm)
        want = s.check_join(x_out, r, r_post)
        assert n.dtype == s.io
        ref.assert_within(n, want, want.abs(), s.io, "n")


@pytest.mark.parametrize("gate", [0, 1, 2, 5, 41, 100])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gamma", [False, True])
def test_norm_step_options(hna, gate, post, gamma):
    for T, C, res, io in ((41, 200, F, BF), (6, 2200, BF, BF)):
        s = Step(T, C, res, io, post=post, gate=gate, gamma=gamma, rs=1.0, bs=2.0, eps=1e-5)
        x_out, n, r, r_post = s.forward(hna.block_norm)
        want = s.check_join(x_out, r, r_post)
        ref.assert_within(n, want, want.abs(), io, "n")
        assert (r_post is None) == (not post)


def test_norm_step_in_place_and_rows_behind(hna):
    s = Step(11, 264, F, F, gate=4)
    ref_out = s.forward(hna.block_norm)
    x, y = s.x.clone(), s.y.clone()
    tail = [torch.full((5, s.C), 7.0, device="cuda") for _ in range(2)]
    x_all, n_all = torch.cat([x, tail[0]]), torch.cat([y, tail[1]])
    r_all = torch.full((16,), 7.0, device="cuda")
    s.x, s.y = x_all[:11], n_all[:11]
    s.forward(hna.block_norm, x_out=x_all[:11], n=n_all[:11], r=r_all[:11])
    assert torch.equal(x_all[:11], ref_out[0]) and torch.equal(n_all[:11], ref_out[1])
    assert torch.equal(r_all[:11], ref_out[2])
    assert bool((x_all[11:] == 7).all()) and bool((n_all[11:] == 7).all()) and bool((r_all[11:] == 7).all())


def test_norm_step_zero_and_non_finite_rows(hna):
    """A row of zeros with eps 0 gives zeros (and no NaN in its gradients); a bad row stays by itself."""
    for C in (72, 1496, 4096):
        s = Step(6, C, F, F, eps=0.0, gate=6)
        s.x[1] = 0
        s.y[1] = 0
        s.y[3] = 0                                 # the block's norm alone is empty
        s.x[4, 5] = NAN
        s.y[5, 7] = float("inf")
        x_out, n, r, r_post = s.forward(hna.block_norm)
        assert r[1] == 0 and r_post[1] == 0 and r_post[3] == 0
        assert not n[1].any() and not x_out[1].any()
        good = [0, 1, 2, 3]
        assert bool(torch.isfinite(n[good]).all()) and bool(torch.isnan(n[4]).all()) and bool(torch.isnan(x_out[5, 7]))
        t = Step(6, C, F, F, eps=0.0, gate=6)
        t.x, t.y = s.x[good].clone(), s.y[good].clone()
        clean = t.forward(hna.block_norm)
        assert torch.equal(clean[0], x_out[good]) and torch.equal(clean[1], n[good])
        t.T, t.dn, t.dx_out = 4, s.dn[good].clone(), s.dx_out[good].clone()
        t.gate_tokens = 4
        got = t.backward(hna, clean[0], clean[2], clean[3])
        t.check_backward(got, clean[0], clean[2], clean[3])


def test_norm_step_extremes(hna):
    """Values whose squares stay finite in fp32, tiny ones with eps, and one huge channel."""
    s = Step(4, 512, F, F, eps=1e-6)
    s.x[0] *= 1e15
    s.y[1] *= 1e-18
    s.x[2, 3] = 1e12
    x_out, n, r, r_post = s.forward(hna.block_norm)
    want = s.check_join(x_out, r, r_post)
    ref.assert_within(n, want, want.abs(), F, "n")


def test_no_tokens(hna):
    s = Step(0, 64, F, BF)
    x_out, n, r, r_post = s.forward(hna.block_norm)
    assert x_out.shape == n.shape == (0, 64) and r.shape == r_post.shape == (0,)
    got = s.backward(hna, x_out, r, r_post)
    torch.cuda.synchronize()
    assert not got["dgamma"].any() and not got["dgamma_post"].any()
    q, sc = hna.quant_rows(torch.empty(0, 40, device="cuda"))
    assert q.shape == (0, 48)
    w = torch.zeros(8, 48, dtype=torch.int8, device="cuda")
    assert hna.quant_matmul(q, sc, w, torch.ones(8, device="cuda")).shape == (0, 8)


# ---------------------------------------------------------------------------- backward
@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("res,io", TYPES)
def test_backward_sizes_and_types(hna, T, C, res, io):
    print(f"backward T={T} C={C} {res} {io}", flush=True)
    for kw in (dict(gate=3), dict(y=False), dict(post=False)):
        s = Step(T, C, res, io, **kw)
        x_out, _, r, r_post = s.forward(hna.block_norm)
        got = s.backward(hna, x_out, r, r_post)
        s.check_backward(got, x_out, r, r_post)


@pytest.mark.parametrize("T,C,gate", [
    (2600, 64, 0), (2600, 64, 1), (2600, 64, 2), (2600, 64, 3), (2600, 64, 7), (2600, 64, 800), (2600, 64, 2599),
    (2600, 64, 2600), (5000, 136, 1300), (5000, 136, 6), (9000, 40, 9), (9000, 40, 4096), (1500, 2056, 700),
    (1500, 2056, 1), (1500, 2056, 2), (700, 5000, 333), (300, 8208, 7), (300, 8208, 299)])
@pytest.mark.parametrize("post", [False, True])
def test_backward_gates(hna, T, C, gate, post):
    """Gate rows of every length: within a workgroup's rows, across several, a last one cut short."""
    print(f"backward gates T={T} C={C} gate={gate} post={post}", flush=True)
    s = Step(T, C, BF, F, gate=gate, post=post)
    x_out, _, r, r_post = s.forward(hna.block_norm)
    got = s.backward(hna, x_out, r, r_post)
    s.check_backward(got, x_out, r, r_post)
    again = s.backward(hna, x_out, r, r_post)
    for k in got:
        assert got[k] is None or torch.equal(got[k], again[k]), k       # a fixed order of summation


def test_backward_long_column_sums(hna):
    s = Step(40000, 24, F, F, gate=20000)
    x_out, _, r, r_post = s.forward(hna.block_norm)
    s.check_backward(s.backward(hna, x_out, r, r_post), x_out, r, r_post)


def test_backward_optional_gradients(hna):
    s = Step(50, 136, F, BF, gate=8)
    x_out, _, r, r_post = s.forward(hna.block_norm)
    full = s.backward(hna, x_out, r, r_post)
    got = s.backward(hna, x_out, r, r_post, dx_out=None)
    s.check_backward(got, x_out, r, r_post, dx_out=False)
    got = s.backward(hna, x_out, r, r_post, dn=None)
    assert got["dgamma"] is None
    s.check_backward(got, x_out, r, r_post, dn=False)
    got = s.backward(hna, x_out, r, r_post, want_dy=False)
    assert got["dy"] is None
    for k in ("dx", "dgamma", "dgamma_post", "dgate"):
        assert torch.equal(got[k], full[k])
    # in place: dx over dx_out, dy over dn; and the block's own gradients left out
    dn, dx_out = s.dn.clone(), s.dx_out.clone()
    got = s.backward(hna, x_out, r, r_post, dn=dn, dx_out=dx_out, dx=dx_out, dy=dn)
    for k in full:
        assert torch.equal(got[k], full[k]), k
    y = s.y.clone()
    got = s.backward(hna, x_out, r, r_post, y=y, dy=y)
    for k in full:
        assert torch.equal(got[k], full[k]), k
    got = s.backward(hna, x_out, r, None, y=None, gamma_post=None, gate=None, gate_tokens=None, want_dy=False)
    assert torch.equal(got["dx"], full["dx"]) and torch.equal(got["dgamma"], full["dgamma"])


def test_backward_gate_without_y(hna):
    """A gate whose gradient is not wanted: dy = block_scale gate d needs no y."""
    for gate in (1, 7, 50):
        s = Step(50, 520, F, BF, post=False, gate=gate)
        x_out, _, r, _ = s.forward(hna.block_norm)
        full = s.backward(hna, x_out, r, None)
        got = s.backward(hna, x_out, r, None, y=None)
        assert got["dgate"] is None
        for k in ("dx", "dy", "dgamma"):
            assert got[k].dtype == full[k].dtype
        s.check_backward({**got, "dgate": full["dgate"]}, x_out, r, None)


def test_c_calls_with_outputs_left_out(hna):
    """Every optional output of the C calls left out by itself: the others as with it, bit for bit."""
    import ctypes
    L = hna.lib()
    s = Step(37, 520, F, BF, gate=8)
    x_out, n, r, r_post = s.forward(hna.block_norm)
    _, q, sc, _, _ = s.forward(hna.block_norm_quant)
    dims = hna.hna_norm_dims(37, 8, 520, 1, 0)
    st = torch.cuda.current_stream().cuda_stream
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    head = [ctypes.byref(dims), at(s.x), at(s.y), at(s.gate), at(s.gamma), at(s.gamma_post), s.rs, s.bs, s.eps]
    blank = lambda ts: [torch.full_like(t, 77) for t in ts]  # noqa: E731
    for ref_out, call, needed in (((x_out, n, r, r_post), L.hna_block_norm, 1),
                                  ((x_out, q, sc, r, r_post), L.hna_block_norm_quant, 3)):
        for skip in range(needed, len(ref_out)):
            out = blank(ref_out)
            assert call(*head, *[None if i == skip else at(t) for i, t in enumerate(out)], st) == 0, hna.last_error()
            for i, t in enumerate(out):
                assert torch.equal(t, ref_out[i]) if i != skip else bool((t == 77).all())
    full = s.backward(hna, x_out, r, r_post)
    ws = torch.empty(hna.block_norm_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    names = ("dx", "dy", "dgamma", "dgamma_post", "dgate")
    for only in (False, True):
        for k in range(5):
            out = blank([full[x] for x in names])
            give = [at(t) if (i == k) == only else None for i, t in enumerate(out)]
            rc = L.hna_block_norm_backward(ctypes.byref(dims), at(s.dn), at(s.dx_out), at(x_out), at(s.y), at(s.gate),
                                           at(s.gamma), at(s.gamma_post), at(r), at(r_post), s.rs, s.bs, *give,
                                           at(ws), ws.numel(), st)
            assert rc == 0, hna.last_error()
            for i, t in enumerate(out):
                assert torch.equal(t, full[names[i]]) if give[i] else bool((t == 77).all()), (only, k, i)


def test_backward_against_differences(hna):
    """<gradient, v> against central differences of the 64-bit forward along v: the differences' own
    error is h^2 times third derivatives (h = 1e-4, values of order 1), the kernel's that of its bound."""
    s = Step(20, 320, F, F, gate=6)
    x_out, _, r, r_post = s.forward(hna.block_norm)
    got = s.backward(hna, x_out, r, r_post)
    dn, dx_out = wide(s.dn), wide(s.dx_out)
    names = ("x", "y", "gamma", "gamma_post", "gate")

    def loss(t):
        h, _, _ = ref.join(t["x"], t["y"], t["gamma_post"], t["gate"], s.gate_tokens, s.rs, s.bs, s.eps)
        return (ref.norm(h, t["gamma"], s.eps)[0] * dn).sum() + (h * dx_out).sum()

    t = {k: wide(getattr(s, k)) for k in names}
    g = gen(99)
    for k in names:
        v = torch.randn(t[k].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        diff = (loss({**t, k: t[k] + h * v}) - loss({**t, k: t[k] - h * v})) / (2 * h)
        have = (got["d" + k].double() * v).sum()
        size = (got["d" + k].double() * v).abs().sum()
        assert abs(float(have - diff)) <= 1e-5 * float(size), k


# ---------------------------------------------------------------------------- 8-bit rows
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 16), (70, 100), (9, 520), (4, 1024), (3, 1031), (2, 4096),
                                    (2, 4100), (2, 9000), (2, 14336), (2, 16384), (2, 16400), (1, 131056)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_quant_rows_exact(hna, rows, K, dtype):
    x = randn(gen(rows + K), rows, K, dtype=dtype, scale=3.0)
    if rows > 2:
        x[1] = 0
    q, scale = hna.quant_rows(x)
    want, s = ref.quant(x.double())
    assert q.shape == (rows, hna.quant_pitch(K)) and not q[:, K:].any()
    assert torch.equal(q[:, :K].double(), want)
    ref.assert_within(scale, s, s, F, "scale", 0)


@pytest.mark.parametrize("dtype", [BF, F])
def test_quant_rows_ties(hna, dtype):
    """Every half: rows whose largest value makes k + 1/2 exact (ties to even), at sizes of both ends of
    the type's range; and fp32's neighbours of a half, on either side of it."""
    k = torch.arange(-127, 127, dtype=torch.float64, device="cuda") + 0.5
    for e in (-120, -60, 0, 60, 118):
        x = torch.cat([k, torch.tensor([127.0], device="cuda", dtype=torch.float64)])
        x = torch.stack([x, 2 * x]) * 2.0 ** e
        q, scale = hna.quant_rows(x.to(dtype))
        want, s = ref.quant(x.to(dtype).double())
        assert torch.equal(q[:, :255].double(), want), e
        ref.assert_within(scale, s, s, F, "scale", 0)
    if dtype == F:
        top = 1.2345678
        half = ((k.abs() * float(torch.tensor(top)) / 127).float())
        x = torch.stack([torch.nextafter(half, half + 1), half, torch.nextafter(half, half - 1)])
        x = torch.cat([x, torch.full((3, 1), top, device="cuda")], 1)
        q, _ = hna.quant_rows(x)
        assert torch.equal(q[:, :255].double(), ref.quant(x.double())[0])


def test_quant_rows_smallest_largest_and_non_finite(hna):
    x = randn(gen(5), 8, 40)
    x[0] *= 1e-40 / x[0].abs().max()               # subnormal rows
    x[1] = 0
    x[1, 3] = 1e-45
    x[2] *= 3.4e38 / x[2].abs().max()
    x[3, 4] = NAN
    x[4, 4] = float("inf")
    x[5, 4] = -float("inf")
    q, scale = hna.quant_rows(x)
    for i in (0, 1, 2, 6, 7):
        want, s = ref.quant(x[i:i + 1].double())
        assert torch.equal(q[i:i + 1, :40].double(), want), i
        assert abs(float(scale[i]) - float(s)) <= max(2.0 ** -24 * float(s), 2.0 ** -150), i
    assert bool(torch.isnan(scale[3:6]).all()) and not q[3:6].any()
    out = hna.quant_matmul(q, scale, q[6:8].clone(), scale[6:8].clone(), dtype=F)
    assert bool(torch.isnan(out[3:6]).all()) and bool(torch.isfinite(out[[0, 1, 6, 7]]).all())


@pytest.mark.parametrize("T,C", [(1, 8), (5, 24), (33, 520), (3, 1024), (2, 1536), (4, 4096), (2, 8200), (2, 16384)])
@pytest.mark.parametrize("res,io", TYPES)
def test_norm_quant(hna, T, C, res, io):
    """n of the same step as 8-bit rows: within half a step, plus what fp32 leaves of 127 n / max|n|
    (two values of 64 roundings each: 127 * 128 * 2^-24 < 0.001); x', r, r_post as without them, bit for bit."""
    s = Step(T, C, res, io, gate=2)
    x_out, q, scale, r, r_post = s.forward(hna.block_norm_quant)
    n = s.check_join(x_out, r, r_post)
    for a, b in zip((x_out, r, r_post), (lambda o: (o[0], o[2], o[3]))(s.forward(hna.block_norm))):
        assert torch.equal(a, b)
    top = n.abs().amax(1)
    ref.assert_within(scale, top / 127, top / 127, F, "scale")
    assert q.shape == (T, hna.quant_pitch(C)) and not q[:, C:].any()
    off = (q[:, :C].double() - 127 * n / top[:, None]).abs()
    assert float(off.max()) <= 0.501
    assert bool((q.abs().amax(1) == 127).all())


def test_norm_quant_zero_and_nan_rows(hna):
    s = Step(3, 64, F, F, post=False, eps=0.0)
    s.x[0] = 0
    s.y[0] = 0
    s.x[1, 2] = NAN
    _, q, scale, r, _ = s.forward(hna.block_norm_quant)
    assert scale[0] == 0 and not q[:2].any() and bool(torch.isnan(scale[1])) and r[0] == 0 and bool(q[2].any())


# --------------------------------------------------------------------------- the product
def int_rows(g, rows, K, lo=-127, hi=128):
    pitch = -(-K // 16) * 16
    q = torch.zeros(rows, pitch, dtype=torch.int8, device="cuda")
    q[:, :K] = torch.randint(lo, hi, (rows, K), generator=g, device="cuda").to(torch.int8)
    return q, torch.rand(rows, generator=g, device="cuda") * 0.01 + 1e-4


def check_product(hna, q, s, w, ws, dtype, out=None):
    got = hna.quant_matmul(q, s, w, ws, dtype=dtype, out=out)
    want = (q.double() @ w.double().t()) * s.double()[:, None] * ws.double()
    # the sum's conversion and two products: 3 roundings
    ref.assert_within(got, want, want.abs(), dtype, f"out {tuple(got.shape)} K={q.shape[1]}", 3)
    return got


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 31, 33, 64, 65, 100, 129, 200, 257, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (5, 33), (32, 64), (33, 200), (64, 1000), (100, 128), (130, 144), (257, 400),
                                 (260, 1040), (513, 272)])
def test_product_sizes(hna, T, N, K):
    print(f"product T={T} N={N} K={K}", flush=True)
    g = gen(T * 1000 + N + K)
    q, s = int_rows(g, T, K)
    w, ws = int_rows(g, N, K)
    for dtype in (BF, F):
        check_product(hna, q, s, w, ws, dtype)


@pytest.mark.parametrize("T,N,K", [(1, 14336, 4096), (1, 4096, 14336), (3, 1000, 131056), (20, 2531, 5000),
                                   (48, 4096, 1024), (150, 4096, 2048), (520, 2056, 1536), (1100, 1030, 528),
                                   (2048, 4096, 1024), (4100, 2050, 272), (300, 9000, 640),
                                   (33000, 520, 144), (20003, 1030, 272), (70000, 261, 130), (9000, 2304, 100),
                                   (66000, 260, 640), (257, 70000, 400)])
def test_product_larger(hna, T, N, K):
    print(f"product T={T} N={N} K={K}", flush=True)
    g = gen(T + N + K)
    q, s = int_rows(g, T, K)
    w, ws = int_rows(g, N, K)
    for dtype in (BF, F):
        check_product(hna, q, s, w, ws, dtype)


@pytest.mark.parametrize("T,N,K", [(1, 4096, 1024), (8, 100, 200), (40, 1000, 512), (100, 8000, 2100), (300, 2531, 1008),
                                   (1100, 1032, 528), (1024, 8192, 272), (20003, 261, 400), (9000, 1284, 130), (5, 33, 90)])
def test_product_pair(hna, T, N, K):
    """Two weight matrices in one launch: each output as the single call's, bit for bit (exact sums,
    the same two products of the scales)."""
    print(f"pair T={T} N={N} K={K}", flush=True)
    g = gen(T + N + K)
    q, s = int_rows(g, T, K)
    w0, s0 = int_rows(g, N, K)
    w1, s1 = int_rows(g, N, K)
    for dtype in (BF, F):
        a, b = hna.quant_matmul_pair(q, s, w0, s0, w1, s1, dtype=dtype)
        assert torch.equal(a, check_product(hna, q, s, w0, s0, dtype))
        assert torch.equal(b, check_product(hna, q, s, w1, s1, dtype))
    out = torch.empty(T, N, device="cuda")
    assert hna.quant_matmul_pair(q, s, w0, s0, w1, s1, out1=out)[1] is out and torch.equal(out, b)


def test_product_largest_sums(hna):
    """Every entry at the ends of 8 bits, -128 too, at the longest K: sums up to 2^31 - 2^18."""
    K = 131056
    for T in (2, 40, 300):
        q = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
        w = torch.full((20, K), -128, dtype=torch.int8, device="cuda")
        w[1] = 127
        one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
        got = hna.quant_matmul(q, one(T), w, one(20), dtype=F)
        assert bool((got[:, 0] == float(128 * 128 * K)).all())
        assert bool((got[:, 1] == float(torch.tensor(-128 * 127 * K, dtype=torch.float64).float())).all())


def test_product_operands_at_the_end_of_their_memory_and_rows_behind(hna):
    """Rows behind T and N of larger buffers are neither read into sums nor written."""
    g = gen(3)
    q, s = int_rows(g, 50, 100)
    w, ws = int_rows(g, 80, 100)
    s[37:], ws[61:] = NAN, NAN
    out = torch.full((50 * 61,), 7.0, device="cuda")
    got = check_product(hna, q[:37], s[:37], w[:61], ws[:61], F, out=out[:37 * 61].view(37, 61))
    assert bool(torch.isfinite(got).all()) and bool((out[37 * 61:] == 7).all())


def test_product_past_32_bit_offsets(hna):
    """Operands and output over 2 GiB and 2^31 elements: checked at their first and last rows."""
    T, N, K = 1 << 20, 2064, 2064
    g = gen(8)
    q = torch.zeros(T, K, dtype=torch.int8, device="cuda")
    rows = torch.tensor([0, 1, 1040383, T - 300, T - 1], device="cuda")
    q[rows] = torch.randint(-127, 128, (5, K), generator=g, device="cuda").to(torch.int8)
    s = torch.ones(T, device="cuda")
    w, ws = int_rows(g, N, K)
    got = hna.quant_matmul(q, s, w, ws)
    want = (q[rows].double() @ w.double().t()) * ws.double()
    ref.assert_within(got[rows], want, want.abs(), BF, "out", 3)
    assert int((got != 0).any(1).sum()) == 5


# ------------------------------------------------------------------ streams, graphs, paths
def test_calls_follow_the_current_stream(hna):
    s = Step(200, 1024, BF, BF, gate=50)
    want = s.forward(hna.block_norm)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    x = s.x.clone()
    with torch.cuda.stream(st):
        for _ in range(8):
            big = big @ big * 1e-3
        s.x.zero_()
        s.x.copy_(x)                               # late on this stream: a launch elsewhere would miss it
        got = s.forward(hna.block_norm)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_step_replays(hna):
    """Forward, 8-bit forward, product and backward in one graph, replayed on new inputs with eager work
    between; every replay equals the eager calls bit for bit."""
    s = Step(96, 520, F, BF, gate=40)
    w, ws = hna.quant_rows(randn(gen(2), 264, 520))
    buf = {}

    def step():
        x_out, n, r, r_post = s.forward(hna.block_norm)
        _, q, sc, _, _ = s.forward(hna.block_norm_quant)
        out = {"x_out": x_out, "n": n, "q": q, "g": hna.quant_matmul(q, sc, w, ws)}
        out.update(s.backward(hna, x_out, r, r_post))
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf = step()
    for rep in range(4):
        s.x.copy_(randn(gen(50 + rep), 96, 520))
        s.dn.copy_(randn(gen(60 + rep), 96, 520, dtype=BF))
        for t in buf.values():
            t.fill_(NAN if t.dtype.is_floating_point else 77)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for k in buf:
            assert torch.equal(buf[k], want[k]), (rep, k)


def test_two_streams_at_once(hna):
    """Two backward passes with their own workspaces at the same time, each as it is alone."""
    steps = [Step(3000, 512, F, BF, gate=100, seed=k) for k in (1, 2)]
    fwd = [s.forward(hna.block_norm) for s in steps]
    alone = [s.backward(hna, f[0], f[2], f[3]) for s, f in zip(steps, fwd)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = []
    for st, s, f in zip(streams, steps, fwd):
        with torch.cuda.stream(st):
            got.append([s.backward(hna, f[0], f[2], f[3]) for _ in range(5)])
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for run in runs:
            for k in want:
                assert torch.equal(run[k], want[k]), k


def test_refused_gpu_arguments(hna):
    x = torch.zeros(8, 64, device="cuda")
    g = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="GPU"):
        hna.block_norm(x, x.cpu(), g)
    with pytest.raises(ValueError, match="contiguous"):
        hna.block_norm(torch.zeros(64, 8, device="cuda").t(), None, g)
    with pytest.raises(hna.HnaError, match="multiple of 8"):
        hna.block_norm(x[:, :60].contiguous(), None, None)
    with pytest.raises(hna.HnaError, match="aligned"):
        hna.quant_rows(torch.zeros(65, device="cuda")[1:].view(1, 64))
    with pytest.raises(hna.HnaError, match="multiple of 16"):
        i8 = torch.zeros(4, 24, dtype=torch.int8, device="cuda")
        hna.quant_matmul(i8, torch.ones(4, device="cuda"), i8, torch.ones(4, device="cuda"))
    with pytest.raises(hna.HnaError, match="workspace"):
        hna.block_norm_backward(x, torch.ones(8, device="cuda"), dn=x, gamma=g,
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("config,T", [(1, 300), (2, 130)])
def test_layer_inputs_feed_the_affinity_pass(hna, config, T):
    """Norm step, 8-bit rows, both products and the affinity pass in a run: r, g, u of the layer with
    8-bit weights against 64 bits, then the scores against the oracle on the same r, g, u."""
    L = synth.make_config_layer(config, T=T, with_x=True)
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) and not k.startswith("group_of") else v) for k, v in L.items()}
    ffn = hna.FfnInputs(dev, eps=0.0)
    y = (dev["a"].reshape(T, -1).float() @ dev["W_o"].float().t())          # the attention output
    got = ffn.run((dev["x_in"] - y), y.bfloat16())
    n, r = ref.norm(got["x_in"].double(), dev["gamma"].double(), 0.0)
    ref.assert_within(got["r"], r, r, F, "r")
    top = n.abs().amax(1)
    ref.assert_within(got["scale"], top / 127, top / 127, F, "scale")
    for k, W in (("g", "W_gate"), ("u", "W_up")):
        wq, ws = ref.quant(dev[W].double())
        # half a step in each of n's entries, against the same 8-bit weights
        want = n @ (wq * ws[:, None]).t()
        slack = 0.501 * (top / 127)[:, None] * (wq * ws[:, None]).abs().sum(1)
        assert bool(((got[k].double() - want).abs() <= slack + ref.half_step(BF) * want.abs() * 1.01 + slack * 2.0 ** -8).all())
        # and near the layer's own pre-activations: a uniform error of one step of max / 127 is max / 440
        # rms; rows of 1024 and more normal values have max <= 5 rms, so W and n each bring <= 1.2%
        rel = float((got[k].double() - dev[k].double()).norm() / dev[k].double().norm())
        assert rel < 0.024, rel
    L2 = dict(L)
    for k in ("r", "g", "u"):
        dev[k] = got[k]
        L2[k] = got[k].cpu()
    scores = hna.affinity_layer(dev)
    torch.cuda.synchronize()
    want = oracle.affinity_layer(L2)
    for key in ("S_fo", "S_add", "S_down"):
        x = scores[key].double().cpu()
        w = torch.as_tensor(want[key])
        assert float((x - w).norm() / w.norm()) <= 1e-2, key
