"""Paths of the norm step and the 8-bit calls that ordinary sizes do not reach: values that one output
must not read, layers of either type, large calls, and calls behind work on another stream."""
import numpy as np
import pytest
import torch

import norm_reference as ref
import oracle
import synth
from test_norm_quant_gpu import BF, F, NAN, Step, hna, wide  # noqa: F401

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
