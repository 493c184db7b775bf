"""The operators around the affinity pass's inputs, case by case, with their plain forms.

A layer's calibration pass reads the rms r of the residual entering a pre-norm, the FFN
pre-activations g and u, and the residual x itself.  The operators here produce them, and carry
gradients back through the same step:

  norm   x' = res_scale x + block_scale gate * N(y; gamma_post),  n = gamma * x' / r,
         r = sqrt(mean(x'^2) + eps): the step between two blocks of a layer, N the rms norm
  bwd    its gradients, from those of n and x'
  lin    out = (q w_q^T) * s[:, None] * w_s: rows of x quantised to 8-bit integers, one scale per
         token, times weights held as 8-bit integers with one scale per channel
  ffn    norm with n quantised at once, then the products with W_gate and W_up: r, g, u of a layer

`own` selects the framework's kernels; otherwise each operator is computed from elementary torch
operations.  x' is rounded to the residual's type and n, r are those of x' as stored.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token between two blocks of a small layer, as in decoding: latency only
        dict(name="norm_token", op="norm", T=1, C=1024, res="bf16", io="bf16", post=False, gate=0, rs=1.0, bs=1.0),
        # a micro-batch of 4 sequences x 1024 tokens with an fp32 residual, norms on both sides of
        # the block and one gate row per sequence
        dict(name="norm_batch", op="norm", T=4096, C=1536, res="f32", io="bf16", post=True, gate=1024, rs=1.0, bs=1.0),
        # calibration tokens of the large layer: a stream of 2 GB
        dict(name="norm_calib", op="norm", T=65536, C=4096, res="bf16", io="bf16", post=False, gate=0, rs=1.0, bs=2.0),
        # a short odd batch in fp32 with one learned gate row for all tokens
        dict(name="bwd_small", op="bwd", T=777, C=1000, res="f32", io="f32", post=True, gate=777, rs=1.0, bs=1.0),
        # a training step's 16 x 1024 tokens, pre-norm only, the block's output scaled by sqrt(L) = 2
        dict(name="bwd_train", op="bwd", T=16384, C=1024, res="f32", io="bf16", post=False, gate=0, rs=1.0, bs=2.0),
        # the large layer with both norms and a gate row per 2048-token sequence
        dict(name="bwd_large", op="bwd", T=32768, C=4096, res="bf16", io="bf16", post=True, gate=2048, rs=1.0, bs=1.0),
        # one token through the large layer's up projection: the weights' bytes
        dict(name="lin_token", op="lin", T=1, K=4096, N=14336, io="bf16", out="bf16"),
        # odd sizes on every side, fp32 in and out
        dict(name="lin_odd", op="lin", T=219, K=1000, N=2531, io="f32", out="f32"),
        # 64 x 1024 calibration tokens through a gate projection
        dict(name="lin_calib", op="lin", T=65536, K=1536, N=4096, io="bf16", out="bf16"),
        # the large layer's down projection
        dict(name="lin_large", op="lin", T=16384, K=14336, N=4096, io="bf16", out="bf16"),
        # a few decoded tokens into an FFN
        dict(name="ffn_few", op="ffn", T=8, C=1024, I=4096, res="bf16", post=False),
        # a prefill of the large layer into its FFN, norms on both sides, fp32 residual
        dict(name="ffn_large", op="ffn", T=8192, C=4096, I=14336, res="f32", post=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "bwd", "lin", "ffn"])
    if op in ("norm", "bwd"):
        C = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, min(65536, (65536 if op == "norm" else 32768) * 4096 // C))
        gate = rng.choice([0, 0, 1, T, _log(rng, 1, T)])
        res, io = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
        if "f32" in (res, io):
            T = max(1, T // 2)
            gate = min(gate, T)
        return dict(op=op, T=T, C=C, res=res, io=io, post=rng.random() < 0.5, gate=gate,
                    rs=rng.choice([1.0, 1.0, 0.5]), bs=rng.choice([1.0, 2.0]))
    if op == "lin":
        K, N = _log(rng, 32, 14336), _log(rng, 32, 14336)
        T = _log(rng, 1, min(65536, 16384 * 14336 // max(K, N), 16384 * 14336 * 4096 // (N * K)))
        io, out = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        if "f32" in (io, out):
            T = max(1, T // 2)
        return dict(op=op, T=T, K=K, N=N, io=io, out=out)
    C, I = 8 * _log(rng, 8, 512), _log(rng, 32, 14336)
    T = _log(rng, 1, min(16384, 8192 * 14336 // I))
    return dict(op=op, T=T, C=C, I=I, res=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5)


_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _size(t):
    return 2 if t == "bf16" else 4


def work(case):
    op, T = case["op"], case["T"]
    if op == "lin":
        K, N = case["K"], case["N"]
        return {"bytes": T * K * _size(case["io"]) + N * K + 4 * N + T * N * _size(case["out"]) + 4 * T, "flops": 2 * T * N * K}
    C = case["C"]
    if op == "ffn":
        s, I = _size(case["res"]), case["I"]
        small = 4 * C * (2 if case["post"] else 1) + 8 * T
        return {"bytes": T * C * (2 * s + 2) + small + 2 * I * (C + 4) + 2 * T * I * 2, "flops": 4 * T * I * C + 10 * T * C}
    s, i, g = _size(case["res"]), _size(case["io"]), case["gate"]
    gates = -(-T // g) * C * i if g else 0
    small = 4 * C * (2 if case["post"] else 1)
    if op == "norm":
        return {"bytes": T * C * (2 * s + 2 * i) + gates + small + 4 * T * (2 if case["post"] else 1), "flops": 10 * T * C}
    reads_y = bool(case["post"] or g)
    return {"bytes": T * C * (3 * s + 2 * i + (i if reads_y else 0)) + 2 * gates + 2 * small + 4 * T * (2 if case["post"] else 1),
            "flops": 20 * T * C}


# ------------------------------------------------------------------------------------ inputs
def _spread(gen, rows, cols, dtype):
    """Activations: channels of unequal size, a few of them large, as residuals and FFN inputs have."""
    d = gen.device
    size = torch.exp(0.5 * torch.randn(cols, generator=gen, device=d))
    size[torch.randint(cols, (max(1, cols // 512),), generator=gen, device=d)] *= 8.0
    return (torch.randn(rows, cols, generator=gen, device=d) * size).to(dtype)


def _weights(gen, rows, cols):
    """8-bit rows [rows, cols rounded up to 16] with zeros behind cols, and their scales."""
    d = gen.device
    w = torch.randn(rows, cols, generator=gen, device=d) / math.sqrt(cols)
    top = w.abs().amax(1, keepdim=True)
    q = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.int8, device=d)
    q[:, :cols] = torch.round(w * (127.0 / top)).to(torch.int8)
    return q, (top / 127.0).reshape(-1)


def _made(case, seed, device):
    gen = torch.Generator(device=device).manual_seed(int(seed))
    op, T = case["op"], case["T"]
    s = dict(case)
    if op == "lin":
        s["x"] = _spread(gen, T, case["K"], _TYPE[case["io"]])
        s["w"], s["ws"] = _weights(gen, case["N"], case["K"])
        return s
    C = case["C"]
    io = _TYPE[case.get("io", "bf16")]
    s["gamma"] = 1.0 + 0.1 * torch.randn(C, generator=gen, device=device)
    s["gamma_post"] = 1.0 + 0.1 * torch.randn(C, generator=gen, device=device) if case["post"] else None
    s["y"] = _spread(gen, T, C, io)
    s["gate_row"] = None
    if case.get("gate"):
        s["gate_row"] = (0.5 + 0.25 * torch.randn(-(-T // case["gate"]), C, generator=gen, device=device)).to(io)
    s["x"] = _spread(gen, T, C, _TYPE[case["res"]])
    if op == "ffn":
        s["wg"], s["wgs"] = _weights(gen, case["I"], C)
        s["wu"], s["wus"] = _weights(gen, case["I"], C)
    if op == "bwd":
        # what the forward pass kept: x' as stored, r and the block norm's r (fp32)
        s["x_out"], s["r"], s["r_post"] = _join(s, torch.float32)
        del s["x"]
        s["dn"] = torch.randn(T, C, generator=gen, device=device).to(io)
        s["dx_out"] = torch.randn(T, C, generator=gen, device=device).to(_TYPE[case["res"]])
        if not (case["post"] or case.get("gate")):
            s["y"] = None   # the gradients do not need it
    return s


def prepare(case, seed):
    return _made(case, seed, "cuda")


# --------------------------------------------------------------------------------- plain form
def _gates(s, T, wide):
    """The gate row of every token, or None."""
    if s["gate_row"] is None:
        return None
    rows = torch.arange(T, device=s["gate_row"].device) // s["gate"]
    return s["gate_row"].to(wide)[rows]


def _join(s, wide):
    """x' as stored, r, and the block norm's r or None."""
    x, y = s["x"], s["y"].to(wide)
    r_post = None
    if s["gamma_post"] is not None:
        r_post = torch.sqrt((y * y).mean(1) + EPS)
        y = y / r_post[:, None] * s["gamma_post"].to(wide)
    gate = _gates(s, x.shape[0], wide)
    if gate is not None:
        y = y * gate
    out = (s.get("rs", 1.0) * x.to(wide) + s.get("bs", 1.0) * y).to(x.dtype)
    h = out.to(wide)
    return out, torch.sqrt((h * h).mean(1) + EPS), r_post


def _quant(x):
    """Rows as 8-bit integers (in float32) and scales: the nearest integer to 127 x / max|x|, ties to
    even; the quotient in 64 bits, where a value next to a border between two integers needs it."""
    top = x.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(127.0 * x.double() / top.double()), 0.0).float()
    return q, (top.float() / 127.0).reshape(-1)


def _product(q, scale, w, w_scale, out):
    return ((q @ w[:, : q.shape[1]].float().t()) * scale[:, None] * w_scale).to(out)


def _plain(s):
    op, f = s["op"], torch.float32
    if op == "lin":
        q, scale = _quant(s["x"].float())
        return {"out": _product(q, scale, s["w"], s["ws"], _TYPE[s["out"]]), "scale": scale}
    if op == "bwd":
        return _plain_bwd(s)
    x_out, r, r_post = _join(s, f)
    n = x_out.float() / r[:, None] * s["gamma"]
    if op == "norm":
        return {"x_out": x_out, "n": n.to(s["y"].dtype), "r": r, "r_post": r_post}
    q, scale = _quant(n)
    return {"x_out": x_out, "r": r, "scale": scale,
            "g": _product(q, scale, s["wg"], s["wgs"], torch.bfloat16),
            "u": _product(q, scale, s["wu"], s["wus"], torch.bfloat16)}


def _plain_bwd(s):
    f = torch.float32
    io, T = s["dn"].dtype, s["dn"].shape[0]
    inv = 1.0 / s["r"][:, None]
    xh = s["x_out"].float() * inv
    dn = s["dn"].float()
    w = dn * s["gamma"]
    d = s["dx_out"].float() + (w - xh * (w * xh).mean(1, keepdim=True)) * inv
    got = {"dgamma": (dn * xh).sum(0), "dx": (s["rs"] * d).to(s["x_out"].dtype)}
    d = s["bs"] * d
    gate = _gates(s, T, f)
    if s["y"] is not None:
        y = s["y"].float()
        yh = y if s["r_post"] is None else y / s["r_post"][:, None]
        if gate is not None:
            p = yh if s["gamma_post"] is None else yh * s["gamma_post"]
            p = torch.nn.functional.pad(d * p, (0, 0, 0, -T % s["gate"]))
            got["dgate"] = p.view(-1, s["gate"], p.shape[1]).sum(1).to(io)
            d = d * gate
        if s["gamma_post"] is not None:
            got["dgamma_post"] = (d * yh).sum(0)
            w = d * s["gamma_post"]
            d = (w - yh * (w * yh).mean(1, keepdim=True)) / s["r_post"][:, None]
    got["dy"] = d.to(io)
    return got


# ---------------------------------------------------------------------------- the framework's
def _kernels(s):
    import head_neuron_affinity_amd as hna
    op = s["op"]
    if op == "lin":
        q, scale = hna.quant_rows(s["x"])
        return {"out": hna.quant_matmul(q, scale, s["w"], s["ws"], dtype=_TYPE[s["out"]]), "scale": scale}
    if op == "ffn":
        got = hna.ffn_inputs(s["x"], s["gamma"], (s["wg"], s["wgs"]), (s["wu"], s["wus"]), y=s["y"],
                             gamma_post=s["gamma_post"], eps=EPS)
        return {"x_out": got["x_in"], "r": got["r"], "scale": got["scale"], "g": got["g"], "u": got["u"]}
    scales = dict(gamma_post=s["gamma_post"], gate=s["gate_row"], gate_tokens=s["gate"] or None,
                  res_scale=s["rs"], block_scale=s["bs"])
    if op == "norm":
        x_out, n, r, r_post = hna.block_norm(s["x"], s["y"], s["gamma"], eps=EPS, **scales)
        return {"x_out": x_out, "n": n, "r": r, "r_post": r_post}
    got = hna.block_norm_backward(s["x_out"], s["r"], dn=s["dn"], dx_out=s["dx_out"], gamma=s["gamma"],
                                  y=s["y"], r_post=s["r_post"], want_dy=True, **scales)
    return {k: v for k, v in got.items() if v is not None}


def run(state):
    return _kernels(state) if own else _plain(state)


# -------------------------------------------------------------------------------- in 64 bits
def _rms_norm64(v):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _forward64(y, x, gamma_post, gate, s):
    """(y, x) -> x' in 64 bits, from the definition."""
    b = y if gamma_post is None else _rms_norm64(y) * gamma_post
    if gate is not None:
        b = b * gate.repeat_interleave(s["gate"], 0)[: y.shape[0]]
    return s.get("rs", 1.0) * x + s.get("bs", 1.0) * b


def _steps64(v):
    """Rows in whole steps of max|row| / 127, and the step."""
    step = v.abs().amax(-1) / 127.0
    return torch.round(v / step.clamp_min(1e-300)[:, None]), step


def exact(case, seed):
    s = _made(case, seed, "cuda" if torch.cuda.is_available() else "cpu")
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"] == "lin":
        # an exact quotient 127 x / max|x| keeps the ties between two integers where they are
        x = wide["x"]
        top = x.abs().amax(1)
        q = torch.round(127.0 * x / top[:, None])
        out = torch.addmm(torch.zeros(1, dtype=torch.float64, device=x.device), q, wide["w"][:, : case["K"]].t())
        return {"out": out * torch.outer(top / 127.0, wide["ws"]), "scale": top / 127.0}
    post, gate = wide.get("gamma_post"), wide.get("gate_row")
    if case["op"] == "bwd":
        return _exact_bwd(case, s, wide, post, gate)
    x_out = _forward64(wide["y"], wide["x"], post, gate, case).to(s["x"].dtype).double()
    n = _rms_norm64(x_out) * wide["gamma"]
    r = (x_out.square().mean(-1) + EPS).sqrt()
    if case["op"] == "norm":
        r_post = None if post is None else (wide["y"].square().mean(-1) + EPS).sqrt()
        return {"x_out": x_out, "n": n, "r": r, "r_post": r_post}
    q, step = _steps64(n)
    up = lambda w, ws: torch.mm(q, wide[w][:, : case["C"]].t()) * step[:, None] * wide[ws][None]  # noqa: E731
    return {"x_out": x_out, "r": r, "scale": step, "g": up("wg", "wgs"), "u": up("wu", "wus")}


def _exact_bwd(case, s, wide, post, gate):
    """The gradients by differentiating the forward formulas, at the x', r and r_post that are given:
    1 / r of a row moves by -(x' . dx') / (C r^3)."""
    T, C = s["dn"].shape
    h, r, dn = wide["x_out"], wide["r"][:, None], wide["dn"]
    got = {"dgamma": torch.einsum("tc,tc->c", dn, h / r)}
    along = (dn * wide["gamma"] * h).sum(1, keepdim=True)
    d = wide["dx_out"] + dn * wide["gamma"] / r - h * along / (C * r ** 3)
    got["dx"] = case["rs"] * d
    d = case["bs"] * d
    if s["y"] is not None:
        y = wide["y"]
        inv = 1.0 if post is None else 1.0 / wide["r_post"][:, None]
        if gate is not None:
            p = d * y * inv * (1.0 if post is None else post)
            rows = torch.arange(T, device=p.device) // case["gate"]
            got["dgate"] = torch.zeros_like(gate).index_add_(0, rows, p)
            d = d * gate.repeat_interleave(case["gate"], 0)[:T]
        if post is not None:
            got["dgamma_post"] = torch.einsum("tc,tc->c", d, y * inv)
            along = (d * post * y).sum(1, keepdim=True)
            d = d * post * inv - y * along * inv ** 3 / C
    got["dy"] = d
    return got
