"""The gate's sigmoid at every finite bf16 gate.  A block with one nonzero
column has the scale h / 448 in fp32, which shows h before it is rounded to
fewer bits: with up = 1, h = gate * sigmoid(gate), one rounding, and the
quotient another; the sigmoid itself is off by at most 5 * 2^-24 of itself from
2^-126 on, and by less than 2^-126 below."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu


def test_every_gate():
    gates = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    gates = gates[torch.isfinite(gates.float())]
    z = torch.zeros(gates.numel(), 256, dtype=torch.bfloat16)
    z[:, 5], z[:, 128 + 5] = gates, 1.0
    _, s = dg.dg_swiglu_quantize_fp8(z.cuda())
    g = gates.double().numpy()
    p = ref.sigmoid(g)
    want = np.abs(g) * p / 448
    # below the normal range the quotient is off by half of 2^-149 more
    bound = np.where(p >= 2.0 ** -126, 7.01 * 2.0 ** -24 * want, np.abs(g) * 2.0 ** -126 / 448) + 2.0 ** -150
    off = np.abs(s[:, 0].cpu().numpy().astype(np.float64) - want)
    assert (off <= bound).all(), (g[off > bound][:5], off[off > bound][:5], bound[off > bound][:5])
