"""Attention over documents, its gradients and single tokens against the formulas in 64 bits; the bounds
are those of tests/attention_reference.py."""
import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def hna():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import head_neuron_affinity_amd as m
    m.lib()
    return m


def inputs(T, H, G, d, dtype, seed=0, size=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h: torch.randn(T, h, d, generator=gen, device="cuda")  # noqa: E731
    return (r(H) * size).to(dtype), (r(G) * size).to(dtype), r(G).to(dtype), r(H).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def within(got, want, bound, name, rows=None):
    got, off = got.double(), None
    if rows is not None:
        got, want, bound = got[rows], want[rows], bound[rows]
    same = got == want                                       # infinities
    off = torch.where(same, torch.zeros_like(got), (got - want).abs() - bound)
    assert not torch.isnan(off).any(), name
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{name}: {worst:.3e} over its bound"


def check(hna, q, k, v, da, rows, causal=True, scale=None, cap=0.0, slopes=None, group_of_head=None):
    T, H, d = q.shape
    how = dict(causal=causal, scale=scale, cap=cap, slopes=slopes, group_of_head=group_of_head)
    seen, live = ref.seen_by(T, rows, causal)
    sc = d ** -0.5 if scale is None else scale
    fill = lambda *s: torch.full(s, 7.0, dtype=q.dtype, device="cuda")  # noqa: E731
    a, lse = hna.attention(q, k, v, rows, out=fill(T, H, d), lse=torch.full((T, H), 7.0, device="cuda"), **how)
    ea, el, oa, ol = ref.forward(q, k, v, seen, sc, cap, slopes, group_of_head)
    within(a, ea, oa, "a", live)
    within(lse, el, ol, "lse", live)
    G = k.shape[1]
    grads = hna.attention_backward(da, q, k, v, a, lse, rows, dq=fill(T, H, d), dk=fill(T, G, d), dv=fill(T, G, d), **how)
    want = ref.backward(da, q, k, v, a, lse, seen, sc, cap, slopes, group_of_head)
    for name, t in zip(("dq", "dk", "dv"), grads):
        within(t, *want[name], name, live)
    for t in (a, lse, *grads):
        assert (t[~live] == 7).all()                          # tokens of no document are left as they were
    return a, lse, grads


HEADS = [(2, 1, 16), (4, 2, 32), (3, 3, 48), (4, 1, 64), (2, 2, 80), (4, 2, 96), (2, 1, 112), (4, 2, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,G,d", HEADS)
@pytest.mark.parametrize("T", [1, 31, 64, 129, 300])
def test_one_document(hna, T, H, G, d, dtype):
    q, k, v, da = inputs(T, H, G, d, dtype, seed=T + d)
    check(hna, q, k, v, da, None)
    check(hna, q, k, v, da, None, causal=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cap,bias", [(0.0, True), (5.0, False), (30.0, True)])
@pytest.mark.parametrize("H,G,d", [(4, 2, 32), (4, 2, 64), (4, 2, 96), (2, 1, 128)])
def test_documents_prefixes_caps_and_slopes(hna, H, G, d, cap, bias, dtype):
    starts = [0, 5, 5, 90, 250, 251, 600, 700]               # an empty document, one of one token, tokens behind the last
    T = 720
    q, k, v, da = inputs(T, H, G, d, dtype, seed=d, size=3.0)
    rows = hna.attention_rows(T, i32(starts), i32([0, 3, 40, 160, 1, 200, 0]))
    assert torch.equal(rows[700:], torch.full((20, 4), -1, dtype=torch.int32, device="cuda"))
    slopes = slopes_of(H) if bias else None
    check(hna, q, k, v, da, rows, cap=cap, slopes=slopes)
    check(hna, q, k, v, da, hna.attention_rows(T, i32(starts), causal=False), cap=cap, slopes=slopes, scale=0.05)


def test_rows_follow_their_definition(hna):
    starts, prefix, T = [3, 10, 10, 40, 64], [2, 5, 100, -4], 70
    for causal in (True, False):
        rows = hna.attention_rows(T, i32(starts), i32(prefix) if causal else None, causal).tolist()
        for t in range(T):
            docs = [i for i in range(4) if starts[i] <= t < starts[i + 1]]
            if not docs:
                assert rows[t] == [-1] * 4
                continue
            s, e = starts[docs[0]], starts[docs[0] + 1]
            known = s + min(max(prefix[docs[0]], 0), e - s) if causal else e
            see = lambda i: range(s, max(i + 1, known) if causal else e)  # noqa: E731
            assert rows[t][:2] == [see(t).start, see(t).stop]
            by = [i for i in range(s, e) if t in see(i)]
            assert rows[t][2:] == [by[0], by[-1] + 1]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_the_callers_own(hna, dtype):
    """A window of 50 keys, with queries that see nothing and keys that nobody sees."""
    T = 333
    q, k, v, da = inputs(T, 4, 2, 64, dtype, seed=8)
    t = torch.arange(T)
    lo, hi = (t - 49).clamp_min(0), t + 1
    nothing = (t % 7 == 0) | ((t >= 128) & (t < 256))
    hi = torch.where(nothing, lo, hi)
    rows = torch.stack([lo, hi, t, (t + 50).clamp_max(T + 90)], 1).to(torch.int32).cuda()
    a, lse, grads = check(hna, q, k, v, da, rows, slopes=slopes_of(4))
    gone = nothing.cuda()
    assert not a[gone].any() and torch.isinf(lse[gone]).all() and not grads[0][gone].any()
    nobody = rows.clone()
    nobody[:, 1] = nobody[:, 0]
    a, lse, grads = check(hna, q, k, v, da, nobody)
    assert not a.any() and not any(g.any() for g in grads)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_group_maps(hna, dtype):
    """q, k, v as parts of one projection's output; heads of a group not next to each other, a group without heads."""
    T, H, G, d = 210, 6, 3, 48
    gen = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn(T, (H + 2 * G) * d, generator=gen, device="cuda").to(dtype)
    q, k, v = (x.view(T, -1, d) for x in qkv.split([H * d, G * d, G * d], 1))
    da = torch.randn(T, H, d, generator=gen, device="cuda").to(dtype)
    rows = hna.attention_rows(T, i32([0, 100, 210]))
    a, lse, grads = check(hna, q, k, v, da, rows, group_of_head=[2, 0, 2, 2, 0, 2])
    assert not grads[1][:, 1].any() and not grads[2][:, 1].any()
    b, _ = hna.attention(*(t.contiguous() for t in (q, k, v)), rows, group_of_head=[2, 0, 2, 2, 0, 2])
    assert torch.equal(a, b)


def test_many_heads_and_many_tokens(hna):
    q, k, v, da = inputs(70, 128, 2, 16, BF16, seed=1)
    check(hna, q, k, v, da, None)
    q, k, v, da = inputs(2500, 2, 1, 128, BF16, seed=2)
    check(hna, q, k, v, da, hna.attention_rows(2500, i32([0, 1100, 2500]), i32([300, 0])), cap=20.0)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (8.0, True)])
def test_gradients_against_autograd_and_differences(hna, cap, bias):
    T, H, G, d = 150, 4, 2, 32
    q, k, v, da = inputs(T, H, G, d, F32, seed=6, size=1.0)
    slopes = slopes_of(H) if bias else None
    rows = hna.attention_rows(T, i32([0, 60, 150]), i32([10, 0]))
    how = dict(cap=cap, slopes=slopes)
    a, lse = hna.attention(q, k, v, rows, **how)
    grads = hna.attention_backward(da, q, k, v, a, lse, rows, **how)
    seen, _ = ref.seen_by(T, rows)
    leaves = [t.double().requires_grad_(True) for t in (q, k, v)]
    far = (torch.arange(T, device="cuda")[None] - torch.arange(T, device="cuda")[:, None]).abs()
    out = []
    for h in range(H):
        s = leaves[0][:, h] @ leaves[1][:, h * G // H].t() * d ** -0.5
        s = cap * torch.tanh(s / cap) if cap else s
        s = s - slopes[h].double() * far if bias else s
        out.append(torch.softmax(s.masked_fill(~seen, -torch.inf), 1) @ leaves[2][:, h * G // H])
    want = torch.autograd.grad(torch.stack(out, 1), leaves, da.double())
    for x, y in zip(grads, want):
        # fp32: p and dp - D are off by some 50 2^-24; over up to 150 terms of either sign
        assert (x.double() - y).norm() <= 1e-5 * y.norm()
    gen = torch.Generator(device="cuda").manual_seed(7)
    for x, grad in zip((q, k, v), grads):
        way = torch.randn(x.shape, generator=gen, device="cuda")
        loss = []
        for s in (1e-2, -1e-2):
            moved = [t + s * way if t is x else t for t in (q, k, v)]
            loss.append((hna.attention(*moved, rows, **how)[0].double() * da.double()).sum().item())
        along = (grad.double() * way.double()).sum().item()
        # the third derivative's share of a step of 1e-2 is a few 1e-4 of the norms' product; fp32's rounding less
        assert abs((loss[0] - loss[1]) / 2e-2 - along) <= 2e-3 * grad.norm().item() * way.norm().item()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_reach_only_those_that_see_them(hna, value, dtype):
    T, H, G, d = 400, 4, 2, 64
    q, k, v, da = inputs(T, H, G, d, dtype, seed=12)
    starts = i32([0, 70, 190, 390])
    rows = hna.attention_rows(T, starts, i32([0, 20, 0]))
    seen, live = ref.seen_by(T, rows)
    a, lse = hna.attention(q, k, v, rows)
    grads = hna.attention_backward(da, q, k, v, a, lse, rows)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[69, 100, 101, 300, 395]] = True
    touched = (seen & bad[None]).any(1)                       # queries that see a bad key
    for which in ("k", "v"):
        k2, v2 = k.clone(), v.clone()
        (k2 if which == "k" else v2)[bad] = value
        if which == "v":
            v2[bad, :, 5:] = v[bad, :, 5:]                    # some of a row's elements
        b, l2 = hna.attention(q, k2, v2, rows)
        clean = live & ~touched
        assert torch.equal(a[clean], b[clean]) and torch.equal(lse[clean], l2[clean])
        if which == "v":
            assert torch.equal(lse[live], l2[live]) and torch.equal(a[live][..., 5:], b[live][..., 5:])
            assert not torch.isfinite(b[touched & live][..., :5]).any()
        else:
            assert not torch.isfinite(b[touched & live]).all(-1).any() or value == float("inf")
        got = hna.attention_backward(da, q, k2, v2, b, l2, rows)
        assert torch.equal(got[0][clean], grads[0][clean])
        # keys seen only by clean queries keep their gradients
        alone = live & ~(seen & touched[:, None]).any(0)
        assert torch.equal(got[1][alone], grads[1][alone]) and torch.equal(got[2][alone], grads[2][alone])
    q2, da2 = q.clone(), da.clone()
    q2[bad], da2[bad] = value, value
    b, l2 = hna.attention(q2, k, v, rows)
    got = hna.attention_backward(da2, q2, k, v, b, l2, rows)
    ok = live & ~bad
    assert torch.equal(a[ok], b[ok]) and torch.equal(got[0][ok], grads[0][ok])
    alone = live & ~(seen & bad[:, None]).any(0)
    assert torch.equal(got[1][alone], grads[1][alone]) and torch.equal(got[2][alone], grads[2][alone])


def test_scores_of_any_size(hna):
    """Scores up to 1e4: the reference moves with them; equal scores average."""
    q, k, v, da = inputs(200, 2, 1, 64, F32, seed=3, size=60.0)
    check(hna, q, k, v, da, None)
    q.zero_()
    a, lse = hna.attention(q, k, v, None, causal=False)
    assert torch.allclose(a[0, 0], v[:, 0].mean(0), atol=1e-5) and torch.allclose(lse, torch.full_like(lse, 200.0).log())


# ------------------------------------------------------------------ single tokens
def check_step(hna, q, k, v, lengths, starts=None, cap=0.0, slopes=None, group_of_head=None):
    B, H, d = q.shape
    G = k.shape[2]
    a, lse = hna.attention_step(q, k, v, i32(lengths), None if starts is None else i32(starts), cap=cap, slopes=slopes,
                                group_of_head=group_of_head)
    for b in range(B):
        n, s0 = lengths[b], 0 if starts is None else starts[b]
        if n <= s0:
            assert not a[b].any() and (lse[b] == -torch.inf).all()
            continue
        at = torch.tensor([n - 1 - s0], device="cuda")
        for h, g in enumerate(ref.groups(H, G, group_of_head)):
            kk, vv = k[b, s0:n, g], v[b, s0:n, g]
            s, _, e = ref.scores(q[b, h][None], kk, at, d ** -0.5, cap, None if slopes is None else slopes[h])
            w, l = ref.softmax(s, torch.ones_like(s, dtype=torch.bool))
            e = e.amax() + (n + 16) * ref.U + ref.U * s.abs().amax()
            want = (w @ vv.double())[0]
            hf = ref.half(q.dtype)
            within(a[b, h], want, (hf + 2 * e) * (w @ vv.double().abs())[0] + hf * want.abs() + 1e-30, f"a {b} {h}")
            within(lse[b, h][None], l, e + 8 * ref.U * l.abs(), f"lse {b} {h}")
    return a, lse


def cache(B, S, H, G, d, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    return r(B, H, d), r(B, S, G, d), r(B, S, G, d)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,G,d", HEADS)
def test_step(hna, H, G, d, dtype):
    q, k, v = cache(5, 700, H, G, d, dtype, seed=d)
    check_step(hna, q, k, v, [1, 700, 33, 0, 257])
    check_step(hna, q, k, v, [31, 640, 129, 5, 32], [0, 600, 128, 5, 7], cap=6.0, slopes=slopes_of(H))


@pytest.mark.parametrize("B,S", [(1, 1), (1, 5000), (3, 20000), (300, 70)])
def test_step_splits(hna, B, S):
    q, k, v = cache(B, S, 8, 2, 64, BF16, seed=S)
    check_step(hna, q, k, v, [S - (17 * b) % S for b in range(B)])


def test_step_many_heads_of_a_group(hna):
    q, k, v = cache(2, 300, 80, 1, 32, BF16)
    check_step(hna, q, k, v, [300, 41], slopes=slopes_of(80))
    q, k, v = cache(2, 300, 80, 2, 32, BF16)
    check_step(hna, q, k, v, [300, 41], group_of_head=[1 if h % 5 else 0 for h in range(80)])


def test_step_reads_nothing_outside_and_takes_strides(hna):
    """A cache with keys and values side by side, whose other rows hold NaNs; lengths past S count as S."""
    B, S, H, G, d = 3, 500, 4, 2, 96
    kv = torch.randn(B, S, 2, G, d, device="cuda").to(BF16)
    q = torch.randn(B, H, d, device="cuda").to(BF16)
    lengths, starts = [500, 77, 300], [0, 3, 130]
    for b in range(B):
        kv[b, lengths[b]:] = float("nan")
        kv[b, :starts[b]] = float("inf")
    k, v = kv[:, :, 0], kv[:, :, 1]
    a, lse = check_step(hna, q, k, v, lengths, starts)
    b, l2 = hna.attention_step(q, k, v, i32([9999, 77, 300]), i32([-4, 3, 130]))
    assert torch.equal(a, b) and torch.equal(lse, l2)
    # one cache for all sequences
    a, _ = hna.attention_step(q, k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1), i32([500] * 3))
    b, _ = hna.attention_step(q, k[:1].repeat(3, 1, 1, 1), v[:1].repeat(3, 1, 1, 1), i32([500] * 3))
    assert torch.equal(a, b)


def test_step_is_the_last_row_of_attention(hna):
    T, H, G, d = 333, 4, 2, 64
    q, k, v, _ = inputs(T, H, G, d, F32, seed=20)
    how = dict(cap=9.0, slopes=slopes_of(H))
    a, lse = hna.attention(q, k, v, **how)
    b, l2 = hna.attention_step(q[-1:], k[None], v[None], i32([T]), **how)
    assert torch.allclose(a[-1], b[0], atol=1e-5) and torch.allclose(lse[-1], l2[0], atol=1e-5)


# ------------------------------------------------------------------ calls
def test_empty_calls(hna):
    q, k, v, da = inputs(0, 4, 2, 32, BF16)
    a, lse = hna.attention(q, k, v)
    assert a.shape == (0, 4, 32) and lse.shape == (0, 4)
    assert [t.shape[0] for t in hna.attention_backward(da, q, k, v, a, lse)] == [0, 0, 0]
    q, k, v = cache(2, 0, 4, 2, 32, BF16)
    a, lse = hna.attention_step(q, k, v, i32([0, 3]))
    assert not a.any() and (lse == -torch.inf).all()
    q, k, v = cache(0, 8, 4, 2, 32, BF16)
    assert hna.attention_step(q, k, v, i32([]))[0].shape == (0, 4, 32)


def test_repeats_on_two_streams(hna):
    made = []
    for T in (300, 900):
        q, k, v, da = inputs(T, 8, 2, 128, BF16, seed=T)
        rows = hna.attention_rows(T, i32([0, T // 3, T]))
        made.append((q, k, v, da, rows, *cache(2, T, 8, 2, 128, BF16), i32([T, T // 2])))

    def run(q, k, v, da, rows, qs, ks, vs, n):
        a, lse = hna.attention(q, k, v, rows, cap=30.0)
        return (a, lse, *hna.attention_backward(da, q, k, v, a, lse, rows, cap=30.0), *hna.attention_step(qs, ks, vs, n))

    want = [run(*m) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = []
    for _ in range(3):
        for s, m in zip(streams, made):
            with torch.cuda.stream(s):
                got.append(run(*m))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(want[i % 2], y))


def test_captured(hna):
    T, H, G, d = 260, 4, 2, 64
    q, k, v, da = inputs(T, H, G, d, BF16, seed=30)
    starts = i32([0, 100, T])
    rows = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    out = [torch.empty(T, H, d, dtype=BF16, device="cuda"), torch.empty(T, H, device="cuda")]
    grads = [torch.empty(T, x, d, dtype=BF16, device="cuda") for x in (H, G, G)]
    dims = hna.hna_attn_dims(T, H * d, G * d, G * d, H, G, d, hna.HNA_BF16, 1, d ** -0.5, 0.0)
    ws = torch.empty(hna.attention_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    qs, ks, vs = cache(1, 3000, H, G, d, BF16)
    n = i32([2900])
    one = [torch.empty(1, H, d, dtype=BF16, device="cuda"), torch.empty(1, H, device="cuda")]
    sdims = hna.hna_step_dims(1, G * d, G * d, 0, 0, 3000, H, G, d, hna.HNA_BF16, d ** -0.5, 0.0)
    ws2 = torch.empty(hna.attention_step_workspace_bytes(sdims), dtype=torch.uint8, device="cuda")

    def step():
        hna.attention_rows(T, starts, rows=rows)
        hna.attention(q, k, v, rows, out=out[0], lse=out[1])
        hna.attention_backward(da, q, k, v, *out, rows, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
        hna.attention_step(qs, ks, vs, n, out=one[0], lse=one[1], workspace=ws2)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        q.copy_(torch.randn(T, H, d, device="cuda"))
        starts.copy_(i32([0, 50 + 60 * r, T]))
        n.fill_(1000 * r + 1)
        for t in (*out, *grads, *one):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (*out, *grads, *one)]
        fresh = hna.attention_rows(T, starts)
        a, lse = hna.attention(q, k, v, fresh)
        eager = (a, lse, *hna.attention_backward(da, q, k, v, a, lse, fresh), *hna.attention_step(qs, ks, vs, n))
        assert all(torch.equal(x, y) for x, y in zip(replayed, eager)), r
