"""Refusals of the attention and gated-FFN calls, on the CPU: every call below fails validation (or has no
tokens), so nothing is launched; the addresses are never read."""
import ctypes
import os

import pytest
import torch

FAKE = 0x7F0000000000
MIS = FAKE + 4
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def hna():
    import head_neuron_affinity_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libhna.so not built (python -m head_neuron_affinity_amd.build_lib)")
    return m


def ptr(v):
    return vp(v) if v else None


# ------------------------------------------------------------------ gated FFN
def ffn_dims(hna, T=8, hidden=64, I=37, dtype=1):
    return hna.hna_ffn_dims(T, hidden, I, dtype)


def ffn(hna, dm, n=FAKE, wg=FAKE, wu=FAKE, g=FAKE, u=FAKE, h=FAKE):
    return hna.lib().hna_gated_ffn(ctypes.byref(dm) if dm is not None else None, ptr(n), ptr(wg), ptr(wu), ptr(g), ptr(u), ptr(h), None)


def ffn_back(hna, dm, dh=FAKE, n=FAKE, wg=FAKE, wu=FAKE, g=FAKE, u=FAKE, dn=FAKE, dwg=FAKE, dwu=FAKE, ws=FAKE, wsb=1 << 40):
    return hna.lib().hna_gated_ffn_backward(ctypes.byref(dm) if dm is not None else None, ptr(dh), ptr(n), ptr(wg), ptr(wu), ptr(g),
                                            ptr(u), ptr(dn), ptr(dwg), ptr(dwu), ptr(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(T=2 ** 31), -2), (dict(hidden=0), -1), (dict(hidden=60), -2), (dict(hidden=65544), -2),
    (dict(I=0), -1), (dict(I=2 ** 20 + 1), -2), (dict(dtype=2), -1), (dict(T=2 ** 20, I=2 ** 15), -2),
    (dict(T=2 ** 30, hidden=128, I=1), -2)])
def test_ffn_bad_dims(hna, kw, status):
    for call in (ffn, ffn_back):
        assert call(hna, ffn_dims(hna, **kw)) == status and hna.last_error() != ""
    assert hna.gated_ffn_workspace_bytes(ffn_dims(hna, **kw)) == 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(n=0), -1, "n is NULL"), (dict(n=MIS), -3, "n is not"), (dict(wg=0), -1, "W_gate is NULL"), (dict(wu=MIS), -3, "W_up is not"),
    (dict(g=MIS), -3, "g is not"), (dict(u=MIS), -3, "u is not"), (dict(h=MIS), -3, "h is not"), (dict(g=0, u=0, h=0), -1, "no output")])
def test_ffn_bad_arguments(hna, kw, status, word):
    assert ffn(hna, ffn_dims(hna), **kw) == status and word in hna.last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(dh=0), -1, "dh is NULL"), (dict(g=0), -1, "g is NULL"), (dict(u=MIS), -3, "u is not"), (dict(n=0), -1, "n is NULL"),
    (dict(wg=0), -1, "W_gate is NULL"), (dict(wu=0), -1, "W_up is NULL"), (dict(dn=MIS), -3, "dn is not"),
    (dict(dwg=0), -1, "wanted together"), (dict(dwu=0), -1, "wanted together"), (dict(dwg=MIS), -3, "dW_gate is not"),
    (dict(dn=0, dwg=0, dwu=0), -1, "no gradient"), (dict(ws=0), -1, "workspace is NULL"), (dict(wsb=100), -4, "workspace has")])
def test_ffn_backward_bad_arguments(hna, kw, status, word):
    assert ffn_back(hna, ffn_dims(hna), **kw) == status and word in hna.last_error()


def test_ffn_without_tokens_or_dims(hna):
    assert ffn(hna, None) == -1 and ffn_back(hna, None) == -1
    assert ffn(hna, ffn_dims(hna, T=0), n=0, wg=0, wu=0, g=0, u=0, h=0) == 0
    assert ffn_back(hna, ffn_dims(hna, T=0), dh=0, n=0, wg=0, wu=0, g=0, u=0, dwg=0, dwu=0) == 0
    assert ffn_back(hna, ffn_dims(hna, T=0), dn=0, dwg=FAKE, dwu=0) == -1


def test_ffn_workspace_grows_with_the_call(hna):
    small, large = (hna.gated_ffn_workspace_bytes(ffn_dims(hna, T=T)) for T in (8, 80))
    assert 2 * 8 * 40 * 2 <= small < large


# ------------------------------------------------------------------ attention
def attn_dims(hna, T=8, ld_q=128, ld_k=64, ld_v=64, H=4, G=2, d=32, dtype=1, causal=1, scale=0.1, cap=0.0):
    return hna.hna_attn_dims(T, ld_q, ld_k, ld_v, H, G, d, dtype, causal, scale, cap)


def imap(m):
    return None if m is None else (ctypes.c_int32 * len(m))(*m)


MAP = (0, 0, 1, 1)


def attn(hna, dm, q=FAKE, k=FAKE, v=FAKE, rows=0, slopes=0, m=MAP, a=FAKE, lse=FAKE):
    return hna.lib().hna_attention(ctypes.byref(dm) if dm is not None else None, ptr(q), ptr(k), ptr(v), ptr(rows), ptr(slopes), imap(m), ptr(a), ptr(lse), None)


def attn_back(hna, dm, da=FAKE, q=FAKE, k=FAKE, v=FAKE, a=FAKE, lse=FAKE, rows=0, slopes=0, m=MAP, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, wsb=1 << 40):
    return hna.lib().hna_attention_backward(ctypes.byref(dm) if dm is not None else None, ptr(da), ptr(q), ptr(k), ptr(v), ptr(a), ptr(lse),
                                            ptr(rows), ptr(slopes), imap(m), ptr(dq), ptr(dk), ptr(dv), ptr(ws), wsb, None)


BAD_HEADS = [(dict(H=0), -1), (dict(G=3), -1), (dict(G=0), -1), (dict(d=24), -2), (dict(d=144), -2), (dict(d=0), -1), (dict(dtype=7), -1),
             (dict(H=130, G=2), -2), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1),
             (dict(scale=float("inf")), -1), (dict(cap=-1.0), -1), (dict(cap=float("nan")), -1), (dict(cap=float("inf")), -1),
             (dict(ld_k=56), -1), (dict(ld_v=68), -2), (dict(ld_k=2 ** 20 + 8), -2)]


@pytest.mark.parametrize("kw,status", BAD_HEADS + [(dict(T=-1), -1), (dict(T=2 ** 29), -2), (dict(T=2 ** 31), -2), (dict(ld_q=120), -1), (dict(ld_q=132), -2)])
def test_attention_bad_dims(hna, kw, status):
    for call in (attn, attn_back):
        assert call(hna, attn_dims(hna, **kw)) == status and hna.last_error() != ""
    assert hna.attention_workspace_bytes(attn_dims(hna, **kw)) == 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(q=0), -1, "q is NULL"), (dict(k=MIS), -3, "k is not"), (dict(v=0), -1, "v is NULL"), (dict(rows=MIS), -3, "rows is not"),
    (dict(slopes=MIS), -3, "slopes is not"), (dict(a=0), -1, "a is NULL"), (dict(lse=MIS), -3, "lse is not"),
    (dict(m=None), -1, "group map is NULL"), (dict(m=(0, 0, 1, 2)), -1, "outside"), (dict(m=(0, 0, 1, -1)), -1, "outside")])
def test_attention_bad_arguments(hna, kw, status, word):
    assert attn(hna, attn_dims(hna), **kw) == status and word in hna.last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(da=0), -1, "da is NULL"), (dict(lse=0), -1, "lse is NULL"), (dict(a=MIS), -3, "a is not"), (dict(dq=0), -1, "dq is NULL"),
    (dict(dk=MIS), -3, "dk is not"), (dict(dv=0), -1, "dv is NULL"), (dict(rows=MIS), -3, "rows is not"), (dict(m=(0, 0, 1, 5)), -1, "outside"),
    (dict(ws=0), -1, "workspace is NULL"), (dict(ws=MIS), -3, "workspace is not"), (dict(wsb=100), -4, "workspace has")])
def test_attention_backward_bad_arguments(hna, kw, status, word):
    assert attn_back(hna, attn_dims(hna), **kw) == status and word in hna.last_error()


def test_attention_without_tokens_or_dims(hna):
    assert attn(hna, None) == -1 and attn_back(hna, None) == -1
    assert attn(hna, attn_dims(hna, T=0), q=0, k=0, v=0, a=0, lse=0) == 0
    assert attn_back(hna, attn_dims(hna, T=0), da=0, q=0, k=0, v=0, a=0, lse=0, dq=0, dk=0, dv=0) == 0


def test_rows_bad_arguments(hna):
    f = hna.lib().hna_attention_rows
    for args, status in (((-1, 1, FAKE, 0, 1, FAKE), -1), ((8, 0, FAKE, 0, 1, FAKE), -1), ((2 ** 30 + 1, 1, FAKE, 0, 1, FAKE), -2),
                         ((8, 1, 0, 0, 1, FAKE), -1), ((8, 1, FAKE, MIS, 1, FAKE), -3), ((8, 1, FAKE, 0, 1, MIS), -3), ((0, 1, 0, 0, 1, 0), 0)):
        T, n, s, p, c, r = args
        assert f(T, n, ptr(s), ptr(p), c, ptr(r), None) == status, args


# ------------------------------------------------------------------ single tokens
def step_dims(hna, B=2, ld_k=64, ld_v=64, bs_k=6400, bs_v=6400, S=100, H=4, G=2, d=32, dtype=1, scale=0.1, cap=0.0):
    return hna.hna_step_dims(B, ld_k, ld_v, bs_k, bs_v, S, H, G, d, dtype, scale, cap)


def step(hna, dm, q=FAKE, k=FAKE, v=FAKE, lengths=FAKE, starts=0, slopes=0, m=MAP, a=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40):
    return hna.lib().hna_attention_step(ctypes.byref(dm) if dm is not None else None, ptr(q), ptr(k), ptr(v), ptr(lengths), ptr(starts),
                                        ptr(slopes), imap(m), ptr(a), ptr(lse), ptr(ws), wsb, None)


@pytest.mark.parametrize("kw,status", BAD_HEADS + [(dict(B=-1), -1), (dict(S=-1), -1), (dict(S=2 ** 30 + 1), -2), (dict(B=2 ** 21), -2),
                                                   (dict(bs_k=-8), -1), (dict(bs_v=6404), -2)])
def test_step_bad_dims(hna, kw, status):
    assert step(hna, step_dims(hna, **kw)) == status and hna.last_error() != ""
    assert hna.attention_step_workspace_bytes(step_dims(hna, **kw)) == 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(q=0), -1, "q is NULL"), (dict(k=0), -1, "k is NULL"), (dict(v=MIS), -3, "v is not"), (dict(lengths=0), -1, "lengths is NULL"),
    (dict(starts=MIS), -3, "starts is not"), (dict(slopes=MIS), -3, "slopes is not"), (dict(a=0), -1, "a is NULL"), (dict(lse=MIS), -3, "lse is not"),
    (dict(m=(0, 0, 1, 9)), -1, "outside"), (dict(ws=0), -1, "workspace is NULL")])
def test_step_bad_arguments(hna, kw, status, word):
    assert step(hna, step_dims(hna), **kw) == status and word in hna.last_error()


def test_step_workspace_and_empty_calls(hna):
    dm = step_dims(hna, B=1, S=4096)
    need = hna.attention_step_workspace_bytes(dm)
    assert need > 256 and step(hna, dm, wsb=need - 1) == -4 and "workspace has" in hna.last_error()
    assert step(hna, step_dims(hna, B=0), q=0, k=0, v=0, lengths=0, a=0, lse=0) == 0
    assert step(hna, None) == -1


# ------------------------------------------------------------------ the binding's own checks
def test_binding_checks_shapes_types_and_devices(hna):
    bf, f = torch.bfloat16, torch.float32
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        hna.gated_ffn(z(4, 16), z(8, 16), z(8, 16))
    with pytest.raises(ValueError, match="w_up"):
        hna.gated_ffn(z(4, 16), z(8, 16), z(7, 16))
    with pytest.raises(ValueError, match="w_gate: dtype"):
        hna.gated_ffn(z(4, 16), z(8, 16, dtype=f), z(8, 16))
    with pytest.raises(ValueError, match="dh"):
        hna.gated_ffn_backward(z(3, 8), z(4, 16), z(8, 16), z(8, 16), z(4, 8), z(4, 8))
    q, k = z(5, 4, 32), z(5, 2, 32)
    with pytest.raises(ValueError, match="GPU"):
        hna.attention(q, k, k)
    with pytest.raises(ValueError, match="next to each other"):
        hna.attention(z(5, 32, 4).transpose(1, 2), k, k)
    with pytest.raises(ValueError, match="v"):
        hna.attention(q, k, z(5, 1, 32))
    with pytest.raises(ValueError, match="rows"):
        hna.attention(q, k, k, z(5, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="slopes"):
        hna.attention(q, k, k, slopes=z(3, dtype=f))
    with pytest.raises(TypeError):
        hna.attention(q.half(), k.half(), k.half())
    with pytest.raises(ValueError, match="doc_start"):
        hna.attention_rows(4, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        hna.attention_rows(4, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="lengths"):
        hna.attention_step(q, z(5, 9, 2, 32), z(5, 9, 2, 32), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="next to each other"):
        hna.attention_step(q, z(5, 9, 32, 2).transpose(2, 3), z(5, 9, 2, 32), torch.zeros(5, dtype=torch.int32))
