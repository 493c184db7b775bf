"""Paths of the norm step and the 8-bit calls that ordinary sizes do not reach: values that one output
must not read, layers of either type, large calls, and calls behind work on another stream."""
import pytest
import torch

import norm_reference as ref
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
