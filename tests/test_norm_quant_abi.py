"""Refusals of the norm step and the 8-bit calls, on the CPU: every call below fails validation (or has
no rows), so nothing is launched; the addresses are never read."""
import ctypes
import os

import pytest

FAKE = 0x7F0000000000
MIS = FAKE + 4
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def hna():
    import head_neuron_affinity_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libhna.so not built (python -m head_neuron_affinity_amd.build_lib)")
    return m


def dims(hna, T=8, gate_tokens=1, hidden=64, dtype=1, res_dtype=0):
    return hna.hna_norm_dims(T, gate_tokens, hidden, dtype, res_dtype)


def ptr(v):
    return vp(v) if v else None


def norm(hna, dm, quant=False, x=FAKE, y=FAKE, gate=0, gamma=FAKE, gamma_post=0, rs=1.0, bs=1.0, eps=1e-6,
         x_out=FAKE, n=FAKE, q_scale=FAKE, r=FAKE, r_post=0):
    L = hna.lib()
    d = ctypes.byref(dm) if dm is not None else None
    head = [d, ptr(x), ptr(y), ptr(gate), ptr(gamma), ptr(gamma_post), rs, bs, eps, ptr(x_out), ptr(n)]
    if quant:
        return L.hna_block_norm_quant(*head, ptr(q_scale), ptr(r), ptr(r_post), None)
    return L.hna_block_norm(*head, ptr(r), ptr(r_post), None)


BAD_DIMS = [(dict(T=-1), -1), (dict(T=2 ** 31), -2), (dict(hidden=0), -1), (dict(hidden=60), -2),
            (dict(hidden=16392), -2), (dict(dtype=2), -1), (dict(res_dtype=5), -1)]


@pytest.mark.parametrize("kw,status", BAD_DIMS)
@pytest.mark.parametrize("quant", [False, True])
def test_norm_bad_dims(hna, kw, status, quant):
    assert norm(hna, dims(hna, **kw), quant) == status
    assert hna.last_error() != ""
    assert hna.block_norm_workspace_bytes(dims(hna, **kw)) == 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=0), -1, "x is NULL"), (dict(x=MIS), -3, "x is not"), (dict(y=MIS), -3, "y is not"),
    (dict(x_out=0), -1, "x_out is NULL"), (dict(n=MIS), -3, "n is not"), (dict(gamma=MIS), -3, "gamma is not"),
    (dict(gate=MIS), -3, "gate is not"), (dict(r=MIS), -3, "r is not"),
    (dict(eps=-1.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"),
    (dict(r_post=FAKE), -1, "r_post without"),
    (dict(y=0), -1, "without y"), (dict(y=0, x_out=0, gate=FAKE), -1, "without y"),
    (dict(y=0, x_out=0, gamma_post=FAKE), -1, "without y"), (dict(y=0, x_out=0, rs=2.0), -1, "without y"),
    (dict(y=0, x_out=0, n=0, r=0), -1, "no output"),
])
def test_norm_bad_arguments(hna, kw, status, word):
    assert norm(hna, dims(hna), **kw) == status
    assert word in hna.last_error()


def test_norm_null_dims_and_gate_tokens(hna):
    assert norm(hna, None) == -1 and "dims is NULL" in hna.last_error()
    assert norm(hna, dims(hna, gate_tokens=0), gate=FAKE) == -1 and "gate_tokens" in hna.last_error()
    assert norm(hna, dims(hna), quant=True, q_scale=0) == -1 and "q_scale is NULL" in hna.last_error()
    assert norm(hna, dims(hna), quant=True, n=0) == -1 and "q is NULL" in hna.last_error()


def backward(hna, dm, dn=FAKE, dx_out=FAKE, x_out=FAKE, y=FAKE, gate=0, gamma=FAKE, gamma_post=0, r=FAKE,
             r_post=0, dx=FAKE, dy=FAKE, dgamma=FAKE, dgamma_post=0, dgate=0, ws=FAKE, wsb=1 << 40):
    d = ctypes.byref(dm) if dm is not None else None
    return hna.lib().hna_block_norm_backward(
        d, ptr(dn), ptr(dx_out), ptr(x_out), ptr(y), ptr(gate), ptr(gamma), ptr(gamma_post), ptr(r), ptr(r_post),
        1.0, 1.0, ptr(dx), ptr(dy), ptr(dgamma), ptr(dgamma_post), ptr(dgate), ptr(ws), wsb, None)


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_backward_bad_dims(hna, kw, status):
    assert backward(hna, dims(hna, **kw)) == status


@pytest.mark.parametrize("kw,status,word", [
    (dict(dn=0, dx_out=0, dgamma=0), -1, "both NULL"), (dict(dn=0), -1, "dgamma without dn"),
    (dict(x_out=0), -1, "x_out is NULL"), (dict(r=0), -1, "r is NULL"), (dict(dn=MIS), -3, "dn is not"),
    (dict(dgate=FAKE), -1, "dgate without gate"), (dict(dgamma_post=FAKE), -1, "dgamma_post without"),
    (dict(gamma_post=FAKE, y=0), -1, "y is NULL"), (dict(gamma_post=FAKE), -1, "r_post is NULL"),
    (dict(gate=FAKE, dgate=FAKE, y=0), -1, "y is NULL"), (dict(gate=FAKE, dgate=MIS), -3, "dgate is not"),
    (dict(dx=0, dy=0, dgamma=0), -1, "no gradient"), (dict(ws=0), -1, "workspace is NULL"),
    (dict(ws=MIS), -3, "workspace is not"), (dict(wsb=0), -4, "workspace has"),
])
def test_backward_bad_arguments(hna, kw, status, word):
    assert backward(hna, dims(hna), **kw) == status
    assert word in hna.last_error()


def test_backward_workspace_is_checked_to_the_byte(hna):
    for kw in (dict(T=5000, gate_tokens=1), dict(T=5000, gate_tokens=700), dict(T=3, gate_tokens=2 ** 31 - 1)):
        dm = dims(hna, **kw)
        need = hna.block_norm_workspace_bytes(dm)
        assert need > 0
        assert backward(hna, dm, gate=FAKE, dgate=FAKE, wsb=need - 1) == -4


def quant(hna, rows=4, K=64, dtype=1, x=FAKE, q=FAKE, scale=FAKE):
    return hna.lib().hna_quant_rows(rows, K, dtype, ptr(x), ptr(q), ptr(scale), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(K=131057), -2), (dict(rows=2 ** 31), -2), (dict(dtype=3), -1),
    (dict(x=0), -1), (dict(q=0), -1), (dict(scale=0), -1), (dict(x=MIS), -3), (dict(q=MIS), -3), (dict(scale=MIS), -3),
])
def test_quant_rows_refusals(hna, kw, status):
    assert quant(hna, **kw) == status and hna.last_error() != ""


def test_quant_pitch(hna):
    assert [hna.quant_pitch(k) for k in (0, -3, 1, 16, 17, 1000, 131056, 131057)] == [0, 0, 16, 16, 32, 1008, 131056, 0]


def matmul(hna, T=4, N=32, K=64, dtype=1, q=FAKE, qs=FAKE, w=FAKE, ws=FAKE, out=FAKE):
    return hna.lib().hna_quant_matmul(T, N, K, dtype, ptr(q), ptr(qs), ptr(w), ptr(ws), ptr(out), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(K=40), -2), (dict(K=131072), -2), (dict(dtype=2), -1),
    (dict(T=2 ** 30 + 1), -2), (dict(N=2 ** 22 + 1), -2), (dict(T=2 ** 20, N=2 ** 17), -2),
    (dict(q=0), -1), (dict(qs=0), -1), (dict(w=0), -1), (dict(ws=0), -1), (dict(out=0), -1),
    (dict(q=MIS), -3), (dict(w=MIS), -3), (dict(qs=MIS), -3), (dict(ws=MIS), -3), (dict(out=MIS), -3),
])
def test_quant_matmul_refusals(hna, kw, status):
    assert matmul(hna, **kw) == status and hna.last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(N=0), -1), (dict(K=40), -2), (dict(dtype=2), -1), (dict(T=2 ** 20, N=2 ** 17), -2)] + [
    ({k: v}, s) for k in ("q", "qs", "w0", "s0", "w1", "s1", "out0", "out1") for v, s in ((0, -1), (MIS, -3))])
def test_quant_matmul_pair_refusals(hna, kw, status):
    a = dict(T=4, N=32, K=64, dtype=1, q=FAKE, qs=FAKE, w0=FAKE, s0=FAKE, w1=FAKE, s1=FAKE, out0=FAKE, out1=FAKE)
    a.update(kw)
    rc = hna.lib().hna_quant_matmul_pair(a["T"], a["N"], a["K"], a["dtype"], *[ptr(a[k]) for k in (
        "q", "qs", "w0", "s0", "w1", "s1", "out0", "out1")], None)
    assert rc == status and hna.last_error() != ""


def test_no_rows_is_no_work(hna):
    assert norm(hna, dims(hna, T=0), x=0, y=0, x_out=0, r=0) == 0
    assert quant(hna, rows=0, x=0, q=0, scale=0) == 0
    assert matmul(hna, T=0, q=0, qs=0, w=0, ws=0, out=0) == 0


def test_python_refuses_host_tensors_and_bad_shapes(hna):
    import torch
    x = torch.zeros(4, 64)
    g = torch.ones(64)
    for call in (lambda: hna.block_norm(x, x, g), lambda: hna.block_norm_quant(x, x, g),
                 lambda: hna.block_norm_backward(x, torch.ones(4), dn=x, gamma=g),
                 lambda: hna.quant_rows(x),
                 lambda: hna.quant_matmul(torch.zeros(4, 64, dtype=torch.int8), torch.ones(4),
                                          torch.zeros(8, 64, dtype=torch.int8), torch.ones(8))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    bf = x.bfloat16()
    i8 = torch.zeros(4, 64, dtype=torch.int8)
    for call in (lambda: hna.block_norm(x, x[:3], g), lambda: hna.block_norm(x, x, g[:32]),
                 lambda: hna.block_norm(x, x, g.double()), lambda: hna.block_norm(x[0], None, g),
                 lambda: hna.block_norm(x, x, g, gate=x, gate_tokens=2),
                 lambda: hna.block_norm(x, x, g, gate=x[:2], gate_tokens=0),
                 lambda: hna.block_norm(x, x, g, gate=bf[:1]),
                 lambda: hna.block_norm(x, None, g, gate=x[:1]),
                 lambda: hna.block_norm(x, None, g, res_scale=2.0),
                 lambda: hna.block_norm(x, x, g, x_out=bf), lambda: hna.block_norm(x, bf, g, n=x),
                 lambda: hna.block_norm_quant(x, x, g, q=i8[:, :48]),
                 lambda: hna.block_norm_backward(x, torch.ones(4)),
                 lambda: hna.block_norm_backward(x, torch.ones(3), dn=x),
                 lambda: hna.block_norm_backward(x, torch.ones(4), dn=x, gamma_post=g),
                 lambda: hna.block_norm_backward(x, torch.ones(4), dn=x, dgate=x[:1]),
                 lambda: hna.quant_rows(x[0]), lambda: hna.quant_rows(x, q=i8[:2]),
                 lambda: hna.quant_matmul(i8, torch.ones(4), i8[:, :32], torch.ones(4)),
                 lambda: hna.quant_matmul(i8, torch.ones(3), i8, torch.ones(4)),
                 lambda: hna.quant_matmul_pair(i8, torch.ones(4), i8, torch.ones(4), i8[:2], torch.ones(4)),
                 lambda: hna.quant_matmul_pair(i8, torch.ones(4), i8, torch.ones(4), i8, torch.ones(4), out0=torch.ones(4, 4),
                                               out1=torch.ones(4, 4).bfloat16()),
                 lambda: hna.quant_matmul(i8, torch.ones(4), i8, torch.ones(4), out=x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: hna.quant_rows(x.half()), lambda: hna.block_norm(x, x.half(), g),
                 lambda: hna.quant_matmul(i8, torch.ones(4), i8, torch.ones(4), dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("gate_tokens", [None, 4, 5, 2**31, 2**63, 2**64 + 1])
def test_gate_tokens_of_any_size_reach_the_library_whole(hna, gate_tokens):
    """One gate row for all tokens stays that, also where gate_tokens does not fit the struct's 64 bits."""
    import torch
    from head_neuron_affinity_amd import _binding as B
    x = torch.zeros(4, 64)
    assert B._norm_dims(x, torch.float32, x[:1], gate_tokens, "x").gate_tokens == 4


def test_calls_run_with_their_tensors_gpu_current(hna, monkeypatch):
    """Tensors of GPU 1 while GPU 0 is current: the call is made with GPU 1 current, on GPU 1's stream
    (a stand-in for the library records the calls; nothing is launched)."""
    import torch
    from head_neuron_affinity_amd import _binding as B
    now, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.before

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace_bytes"):
                    return 256
                seen.append((name, now[0], args[-1]))
                return 0
            return call

    monkeypatch.setattr(B, "_index_of", lambda *ts: 1)
    monkeypatch.setattr(B, "_current", lambda: now[0])
    monkeypatch.setattr(B, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "device", Device)
    x, g, one = torch.zeros(4, 64), torch.ones(64), torch.ones(4)
    i8 = torch.zeros(4, 64, dtype=torch.int8)
    hna.block_norm(x, x, g, gamma_post=g, gate=x, gate_tokens=1, res_scale=2.0, block_scale=3.0, eps=0.5)
    hna.block_norm_quant(x, x, g, gamma_post=g, gate=x, gate_tokens=1, res_scale=2.0, block_scale=3.0, eps=0.5)
    got = hna.block_norm_backward(x, one, dn=x, dx_out=x, gamma=g, y=x, gamma_post=g, r_post=one, gate=x, gate_tokens=1,
                                  res_scale=2.0, block_scale=3.0, want_dy=True)
    hna.quant_rows(x)
    hna.quant_matmul(i8, one, i8, one, dtype=torch.float32)
    a, b = hna.quant_matmul_pair(i8, one, i8, one, i8, one, dtype=torch.float32)
    assert [s[0] for s in seen] == ["hna_block_norm", "hna_block_norm_quant", "hna_block_norm_backward",
                                    "hna_quant_rows", "hna_quant_matmul", "hna_quant_matmul_pair"]
    assert all(s[1:] == (1, 1001) for s in seen) and now == [0]
    assert all(got[k] is not None for k in got) and a.dtype == b.dtype == torch.float32


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_layer_inputs_ask_for_the_layers_type(hna, monkeypatch, kind):
    """FfnInputs asks for g and u in the type of the layer's weights, ffn_inputs for bf16 unless told
    (the calls of the library are recorded, none is made)."""
    import torch
    from head_neuron_affinity_amd import _binding as B
    dtype = torch.float32 if kind == "fp32" else torch.bfloat16
    asked = []

    def pair(q, s, w0, s0, w1, s1, out0=None, out1=None, dtype=torch.bfloat16):
        asked.append(dtype)
        return torch.empty(4, 8, dtype=dtype), torch.empty(4, 8, dtype=dtype)

    monkeypatch.setattr(B, "quant_rows", lambda w: (torch.zeros(8, 64, dtype=torch.int8), torch.ones(8)))
    monkeypatch.setattr(B, "block_norm_quant", lambda x, y, gamma, **kw: (x, None, None, torch.ones(4), None))
    monkeypatch.setattr(B, "quant_matmul_pair", pair)
    layer = {"gamma": torch.ones(64), "W_gate": torch.zeros(8, 64, dtype=dtype), "W_up": torch.zeros(8, 64, dtype=dtype)}
    x = torch.zeros(4, 64)
    got = hna.FfnInputs(layer).run(x)
    assert got["g"].dtype == got["u"].dtype == dtype
    w = B.quant_rows(None)
    hna.ffn_inputs(x, layer["gamma"], w, w)
    hna.ffn_inputs(x, layer["gamma"], w, w, dtype=torch.float32)
    assert asked == [dtype, torch.bfloat16, torch.float32]
