"""Operators that give a layer's pass its head outputs and its FFN pre-activations, case by case.

The affinity pass reads a [T, H, d], the heads' outputs, and g, u [T, I], the FFN's pre-activations.
The operators here compute them from a layer's q, k, v and from its normed FFN input, carry
gradients back through both, and serve one token at a time:

  attn  a = softmax(mask(cap tanh(scale q k^T / cap) - slope |i - j|)) v and the rows' log-sum-exp:
        tokens of several documents in a row, query i sees the keys rows[i, 0] .. rows[i, 1] - 1
        (its own document up to itself, and the document's prefix)
  abwd  its gradients dq, dk, dv
  step  the same for one token per sequence over a cache of keys and values, from its last key on
  ffn   g = n W_gate^T, u = n W_up^T, h = silu(g) u: g and u, or h, or all three
  fbwd  its gradients dn, dW_gate, dW_up from dh

`own` selects the framework's kernels; otherwise each operator is computed from elementary torch
operations.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt of a small fp32 layer in three documents: latency
        dict(name="attn_small", op="attn", T=256, docs=3, ragged=True, prefix=0.0, H=4, G=2, d=16, cap=0.0, bias=False, io="f32"),
        # calibration tokens, 64 sequences of 1024
        dict(name="attn_calib", op="attn", T=65536, docs=64, ragged=False, prefix=0.0, H=16, G=8, d=128, cap=0.0, bias=False, io="bf16"),
        # one long document with a prefix that all of it sees, capped scores and a distance bias
        dict(name="attn_long", op="attn", T=16381, docs=1, ragged=False, prefix=0.125, H=16, G=8, d=96, cap=30.0, bias=True, io="bf16"),
        # a training step on a few ragged documents with a distance bias
        dict(name="abwd_ragged", op="abwd", T=2047, docs=7, ragged=True, prefix=0.2, H=16, G=8, d=96, cap=0.0, bias=True, io="bf16"),
        # a training step of the large layer, 8 sequences of 2048, capped scores
        dict(name="abwd_train", op="abwd", T=16384, docs=8, ragged=False, prefix=0.0, H=32, G=8, d=128, cap=50.0, bias=False, io="bf16"),
        # one sequence of a small layer, the next token
        dict(name="step_one", op="step", B=1, S=4096, H=16, G=8, d=128, cap=0.0, bias=False, io="bf16"),
        # a batch of sequences of unequal length on the large layer
        dict(name="step_batch", op="step", B=96, S=8192, H=32, G=8, d=128, cap=50.0, bias=True, io="bf16"),
        # one token through the large layer's FFN as it is served: the weights' bytes
        dict(name="ffn_token", op="ffn", T=1, C=4096, I=14336, out="h", io="bf16"),
        # odd sizes in fp32, everything kept for a backward pass
        dict(name="ffn_odd", op="ffn", T=219, C=1000, I=2531, out="all", io="f32"),
        # calibration tokens: the pass reads g and u
        dict(name="ffn_calib", op="ffn", T=65536, C=1536, I=4096, out="gu", io="bf16"),
        # a short odd micro-batch
        dict(name="fbwd_short", op="fbwd", T=333, C=1024, I=2531, io="bf16"),
        # a training step of the large layer
        dict(name="fbwd_large", op="fbwd", T=8192, C=4096, I=14336, io="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


_HEADS = [(4, 2, 16), (16, 8, 128), (16, 8, 96), (32, 8, 128), (8, 8, 64), (12, 4, 80), (6, 1, 48)]


def draw(rng):
    op = rng.choice(["attn", "abwd", "step", "ffn", "fbwd"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("attn", "abwd", "step"):
        H, G, d = rng.choice(_HEADS)
        how = dict(H=H, G=G, d=d, cap=rng.choice([0.0, 0.0, 5.0, 30.0, 50.0]), bias=rng.random() < 0.4, io=io)
        if op == "step":
            B, S = _log(rng, 1, 256), _log(rng, 1, 32768)
            return dict(op=op, B=B, S=min(S, max(1, 96 * 8192 // B)), **how)
        while True:
            case = dict(op=op, T=_log(rng, 1, 65536 if op == "attn" else 16384), docs=_log(rng, 1, 64), ragged=rng.random() < 0.6,
                        prefix=rng.choice([0.0, 0.0, 0.1, 0.5, 1.0]), **how)
            # no more work than the largest listed case (fp32's matrix rate is a sixteenth of bf16's), and room for the plain form's scores
            most = dict(attn=5e11, abwd=1.2e12)[op] / (16 if io == "f32" else 1)
            if work(case)["flops"] <= most and case["docs"] * max(_lengths(case)) ** 2 * H < 2 ** 32:
                return case
    C, I = 8 * _log(rng, 8, 512), _log(rng, 32, 14336)
    most = dict(ffn=1.6e12, fbwd=5.5e12)[op] / (16 if io == "f32" else 1)
    T = _log(rng, 1, max(1, min(65536, int(most / (C * I * (4 if op == "ffn" else 12))))))
    case = dict(op=op, T=T, C=C, I=I, io=io)
    if op == "ffn":
        case["out"] = rng.choice(["gu", "h", "all"])
    return case


_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _size(t):
    return 2 if t == "bf16" else 4


def _lengths(case):
    """Tokens of each document (or keys of each sequence of a step): they follow from the case alone."""
    if case["op"] == "step":
        rng = random.Random("%d of %d" % (case["B"], case["S"]))
        return [case["S"]] + [rng.randint((case["S"] + 1) // 2, case["S"]) for _ in range(case["B"] - 1)]
    T, n = case["T"], case["docs"]
    if case["ragged"]:
        rng = random.Random("%d in %d" % (T, n))
        cuts = [0] + sorted(rng.randint(0, T) for _ in range(n - 1)) + [T]
    else:
        cuts = [T * i // n for i in range(n + 1)]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _prefixes(case):
    return [int(case["prefix"] * n) for n in _lengths(case)]


def work(case):
    op, s = case["op"], _size(case["io"])
    if op in ("ffn", "fbwd"):
        T, C, I = case["T"], case["C"], case["I"]
        if op == "ffn":
            outs = {"gu": 2, "h": 1, "all": 3}[case["out"]]
            return {"bytes": s * (T * C + 2 * I * C + outs * T * I), "flops": 4 * T * I * C}
        return {"bytes": s * (3 * T * I + 2 * T * C + 4 * I * C), "flops": 12 * T * I * C}
    H, G, d = case["H"], case["G"], case["d"]
    if op == "step":
        keys = sum(_lengths(case))
        return {"bytes": s * d * (2 * keys * G + 2 * case["B"] * H) + 4 * case["B"] * (H + 1), "flops": 4 * keys * H * d}
    T = case["T"]
    # query i of a document of n tokens sees max(i + 1, p) keys
    pairs = sum(p * p + (n - p) * (n + p + 1) // 2 for n, p in zip(_lengths(case), _prefixes(case)))
    tokens = 2 * H + 2 * G if op == "attn" else 4 * H + 4 * G
    return {"bytes": s * T * d * tokens + T * (4 * H + 16), "flops": (4 if op == "attn" else 10) * pairs * H * d}


# ------------------------------------------------------------------------------------ inputs
def _heads(gen, tokens, H, d, size, dtype):
    """Projections: dimensions of unequal size, as trained layers have."""
    dev = gen.device
    scale = size * torch.exp(0.3 * torch.randn(H, d, generator=gen, device=dev))
    return (torch.randn(tokens, H, d, generator=gen, device=dev) * scale).to(dtype)


def _made(case, seed, device):
    gen = torch.Generator(device=device).manual_seed(int(seed))
    op, io = case["op"], _TYPE[case["io"]]
    s = dict(case)
    if op in ("ffn", "fbwd"):
        T, C, I = case["T"], case["C"], case["I"]
        size = torch.exp(0.3 * torch.randn(C, generator=gen, device=device))
        s["n"] = (torch.randn(T, C, generator=gen, device=device) * size).to(io)
        s["wg"] = (torch.randn(I, C, generator=gen, device=device) / math.sqrt(C)).to(io)
        s["wu"] = (torch.randn(I, C, generator=gen, device=device) / math.sqrt(C)).to(io)
        if op == "fbwd":
            # what the forward pass kept
            s["g"] = (s["n"].float() @ s["wg"].float().t()).to(io)
            s["u"] = (s["n"].float() @ s["wu"].float().t()).to(io)
            s["dh"] = torch.randn(T, I, generator=gen, device=device).to(io)
        return s
    H, G, d = case["H"], case["G"], case["d"]
    s["scale"] = d ** -0.5
    s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=device) if case["bias"] else None
    lengths = _lengths(case)
    if op == "step":
        B, S = case["B"], case["S"]
        s["q"] = _heads(gen, B, H, d, 1.5, io)
        s["k"] = _heads(gen, B * S, G, d, 1.5, io).view(B, S, G, d)
        s["v"] = _heads(gen, B * S, G, d, 1.0, io).view(B, S, G, d)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=device)
        return s
    T = case["T"]
    s["q"] = _heads(gen, T, H, d, 1.5, io)
    s["k"] = _heads(gen, T, G, d, 1.5, io)
    s["v"] = _heads(gen, T, G, d, 1.0, io)
    # the batch's plan: for each token the keys that its query sees, and the queries that see its key
    n = torch.tensor(lengths, dtype=torch.int64)
    first = torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    last = torch.repeat_interleave(torch.cumsum(n, 0), n)
    prefix = first + torch.repeat_interleave(torch.tensor(_prefixes(case), dtype=torch.int64), n)
    t = torch.arange(T)
    s["rows"] = torch.stack([first, torch.maximum(t + 1, prefix), torch.where(t < prefix, first, t), last], 1).to(torch.int32).to(device)
    # documents side by side, for the plain form: the token in each place, or T where a document has ended
    longest = max(lengths)
    place = torch.arange(longest)[None] + (torch.cumsum(n, 0) - n)[:, None]
    s["place"] = torch.where(torch.arange(longest)[None] < n[:, None], place, T).to(device)
    if op == "abwd":
        # what the forward pass kept, and the gradient of its result
        s["a"], s["lse"] = _plain_attention(s)
        s["da"] = torch.randn(T, H, d, generator=gen, device=device).to(io)
    return s


def prepare(case, seed):
    return _made(case, seed, "cuda")


# --------------------------------------------------------------------------------- plain form
def _side_by_side(s, x, groups):
    """[T, heads, d] as [documents, groups, heads of a group x longest, d] in 32 bits, zeros where a document has ended."""
    n, longest = s["place"].shape
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, 1))[s["place"].reshape(-1)]
    x = x.view(n, longest, groups, -1, x.shape[-1]).permute(0, 2, 3, 1, 4)
    return x.reshape(n, groups, -1, x.shape[-1]).contiguous()


def _in_a_row(s, x, heads):
    """The way back, [T, heads, d]."""
    n, longest = s["place"].shape
    x = x.reshape(n, heads, longest, -1).permute(0, 2, 1, 3).reshape(n * longest, heads, -1)
    out = x.new_zeros(s["T"] + 1, heads, x.shape[-1])
    out[s["place"].reshape(-1)] = x
    return out[: s["T"]].contiguous()


def _scores(s):
    """Masked scores [documents, groups, heads of a group, queries, keys], and the slope of the cap."""
    n, longest = s["place"].shape
    G, r = s["G"], s["H"] // s["G"]
    q, k = _side_by_side(s, s["q"], G), _side_by_side(s, s["k"], G)
    x = ((q @ k.transpose(2, 3)) * s["scale"]).view(n, G, r, longest, longest)
    slope = None
    if s["cap"] > 0:
        t = torch.tanh(x / s["cap"])
        x, slope = s["cap"] * t, 1 - t * t
    at = torch.arange(longest, device=x.device)
    if s["slopes"] is not None:
        x = x - s["slopes"].view(G, r, 1, 1) * (at[:, None] - at[None, :]).abs()
    sees = torch.nn.functional.pad(s["rows"][:, :2], (0, 0, 0, 1))[s["place"]] - s["place"][:, :1, None]
    seen = (at >= sees[..., :1]) & (at < sees[..., 1:])
    return x.masked_fill_(~seen[:, None, None], -math.inf), slope


def _plain_attention(s):
    x, _ = _scores(s)
    n, G, r, L, _ = x.shape
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    lse = _in_a_row(s, top + torch.log(total), s["H"])[..., 0]
    a = (x.view(n, G, r * L, L) @ _side_by_side(s, s["v"], G)) / total.view(n, G, r * L, 1).clamp_min(1e-30)
    return _in_a_row(s, a, s["H"]).to(s["q"].dtype), lse


def _plain_attention_backward(s):
    x, slope = _scores(s)
    n, G, r, L, _ = x.shape
    side = lambda t, groups=s["G"]: _side_by_side(s, t, groups)  # noqa: E731
    da = side(s["da"])
    p = torch.exp(x - side(s["lse"][..., None]).view(n, G, r, L, 1))
    del x
    dv = p.view(n, G, r * L, L).transpose(2, 3) @ da
    along = (da * side(s["a"])).sum(-1).view(n, G, r, L, 1)
    ds = p * ((da @ side(s["v"]).transpose(2, 3)).view(n, G, r, L, L) - along)
    ds = (ds if slope is None else ds * slope).view(n, G, r * L, L) * s["scale"]
    dq, dk = ds @ side(s["k"]), ds.transpose(2, 3) @ side(s["q"])
    t = s["q"].dtype
    return {"dq": _in_a_row(s, dq, s["H"]).to(t), "dk": _in_a_row(s, dk, G).to(t), "dv": _in_a_row(s, dv, G).to(t)}


def _plain_step(s):
    B, S, G, d = s["k"].shape
    k, v = (t.float().transpose(1, 2).contiguous() for t in (s["k"], s["v"]))
    x = (s["q"].float().view(B, G, -1, d) @ k.transpose(2, 3)) * s["scale"]
    if s["cap"] > 0:
        x = s["cap"] * torch.tanh(x / s["cap"])
    at, last = torch.arange(S, device=x.device), s["lengths"].view(B, 1, 1, 1) - 1
    if s["slopes"] is not None:
        x = x - s["slopes"].view(G, -1, 1) * (last - at)
    x = x.masked_fill_(at > last, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    a = (x @ v) / total.clamp_min(1e-30)
    return {"a": a.view(B, -1, d).to(s["q"].dtype), "lse": (top + torch.log(total)).view(B, -1)}


def _plain(s):
    op = s["op"]
    if op == "attn":
        a, lse = _plain_attention(s)
        return {"a": a, "lse": lse}
    if op == "abwd":
        return _plain_attention_backward(s)
    if op == "step":
        return _plain_step(s)
    t = s["n"].dtype
    n, wg, wu = s["n"].float(), s["wg"].float(), s["wu"].float()
    if op == "ffn":
        g, u = n @ wg.t(), n @ wu.t()
        got = {"g": g.to(t), "u": u.to(t)} if s["out"] != "h" else {}
        if s["out"] != "gu":
            got["h"] = (g / (1 + torch.exp(-g)) * u).to(t)
        return got
    g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
    sig = 1 / (1 + torch.exp(-g))
    dg, du = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig
    return {"dn": (dg @ wg + du @ wu).to(t), "dwg": (dg.t() @ n).to(t), "dwu": (du.t() @ n).to(t)}


# ---------------------------------------------------------------------------- the framework's
def _kernels(s):
    import head_neuron_affinity_amd as hna
    op = s["op"]
    if op == "ffn":
        g, u, h = hna.gated_ffn(s["n"], s["wg"], s["wu"], want_gu=s["out"] != "h", want_h=s["out"] != "gu")
        return {k: v for k, v in (("g", g), ("u", u), ("h", h)) if v is not None}
    if op == "fbwd":
        dn, dwg, dwu = hna.gated_ffn_backward(s["dh"], s["n"], s["wg"], s["wu"], s["g"], s["u"])
        return {"dn": dn, "dwg": dwg, "dwu": dwu}
    how = dict(scale=s["scale"], cap=s["cap"], slopes=s["slopes"])
    if op == "attn":
        a, lse = hna.attention(s["q"], s["k"], s["v"], s["rows"], **how)
        return {"a": a, "lse": lse}
    if op == "abwd":
        dq, dk, dv = hna.attention_backward(s["da"], s["q"], s["k"], s["v"], s["a"], s["lse"], s["rows"], **how)
        return {"dq": dq, "dk": dk, "dv": dv}
    a, lse = hna.attention_step(s["q"], s["k"], s["v"], s["lengths"], **how)
    return {"a": a, "lse": lse}


def run(state):
    return _kernels(state) if own else _plain(state)


# -------------------------------------------------------------------------------- in 64 bits
def _softmax64(q, k, lo, hi, at, case, slopes):
    """Weights, log-sum-exp and the cap's slope of one head: q [n, d] at places `at`, k [m, d], keys lo <= j < hi seen."""
    z = q @ k.t() * case["d"] ** -0.5
    bent = torch.ones((), dtype=z.dtype, device=z.device)
    if case["cap"] > 0:
        bent = torch.cosh((z / case["cap"]).clamp(-300, 300)).pow(-2)
        z = torch.tanh(z / case["cap"]) * case["cap"]
    j = torch.arange(k.shape[0], device=z.device)
    if slopes is not None:
        z = z - slopes * (j[None] - at[:, None]).abs().double()
    z = torch.where((j[None] >= lo[:, None]) & (j[None] < hi[:, None]), z, -math.inf)
    lse = torch.logsumexp(z, 1)
    return torch.exp(z - lse[:, None]), lse, bent


def exact(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    s = _made(case, seed, dev)
    op = case["op"]
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op in ("ffn", "fbwd"):
        if op == "ffn":
            g, u = torch.mm(wide["n"], wide["wg"].t()), torch.mm(wide["n"], wide["wu"].t())
            got = {} if case["out"] == "h" else {"g": g, "u": u}
            return got if case["out"] == "gu" else {**got, "h": torch.sigmoid(g) * g * u}
        # by differentiating h = silu(g) u at the g and u that are given
        g, u = wide["g"].requires_grad_(True), wide["u"].requires_grad_(True)
        dg, du = torch.autograd.grad(torch.nn.functional.silu(g) * u, (g, u), wide["dh"])
        back = torch.mm(torch.cat([dg, du], 1), torch.cat([wide["wg"], wide["wu"]], 0))
        return {"dn": back, "dwg": torch.mm(dg.t(), wide["n"]), "dwu": torch.mm(du.t(), wide["n"])}
    H, G, d = case["H"], case["G"], case["d"]
    lengths, heads = _lengths(case), range(H)
    slope = lambda h: None if s["slopes"] is None else wide["slopes"][h]  # noqa: E731
    if op == "step":
        a, lse = torch.empty_like(wide["q"]), torch.empty(case["B"], H, dtype=torch.float64, device=dev)
        for b, n in enumerate(lengths):
            one = torch.tensor([n - 1], device=dev)
            for h in heads:
                p, lse[b, h], _ = _softmax64(wide["q"][b, h][None], wide["k"][b, :n, h * G // H], one * 0, one + 1, one, case, slope(h))
                a[b, h] = (p @ wide["v"][b, :n, h * G // H])[0]
        return {"a": a, "lse": lse}
    out = {x: torch.zeros_like(wide[x]) for x in "qkv"}
    a, lse = torch.zeros_like(wide["q"]), torch.zeros(case["T"], H, dtype=torch.float64, device=dev)
    first = 0
    for n, p in zip(lengths, _prefixes(case)):
        here = slice(first, first + n)
        at = torch.arange(n, device=dev)
        for h in heads if n else ():
            x = h * G // H
            q, k, v = wide["q"][here, h], wide["k"][here, x], wide["v"][here, x]
            w, lse[here, h], bent = _softmax64(q, k, 0 * at, torch.clamp(at + 1, min=p), at, case, slope(h))
            if op == "attn":
                a[here, h] = w @ v
                continue
            da = wide["da"][here, h]
            out["v"][here, x] += w.t() @ da
            dw = da @ v.t()
            dz = w * (dw - (w * dw).sum(1, keepdim=True)) * bent * d ** -0.5
            out["q"][here, h] = dz @ k
            out["k"][here, x] += dz.t() @ q
        first += n
    return {"a": a, "lse": lse} if op == "attn" else {"d" + x: out[x] for x in "qkv"}
