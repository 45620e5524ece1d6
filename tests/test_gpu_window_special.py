"""Windowed attention of keys that are not numbers: the rows that see one say so
in out and lse, the others keep their results."""

import math

import pytest
import torch

import oracle
from sequence_exact_attention_gb300 import binding

from helpers import assert_close

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_visible_nan_reaches_out_and_lse(dtype, D, packed):
    """Key 70 of 400 is NaN: rows 70 to 70 + window - 1 see it, each with the
    NaN of its scores in out and in lse (every row sees itself, so -inf, which
    says that a row saw no key, is nobody's lse)."""
    S, window, n_sink, at = 400, 150, 3, 70
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(D)
    q, k, v = (torch.randn(1, S, h, D, generator=g).to(tdt) for h in (4, 2, 2))
    want, want_l = oracle.window_attention(q, k, v, window, n_sink, 1 / math.sqrt(D))
    k[:, at] = float("nan")
    qd, kd, vd = (t.to(DEV) for t in (q, k, v))
    if packed:
        cu = torch.tensor([0, S], dtype=torch.int32, device=DEV)
        out, lse = binding.ring_attn_fwd_window_varlen(qd[0], kd[0], vd[0], cu, S, 1, window, n_sink)
        out, lse = out[None], lse[None]
    else:
        out, lse = binding.ring_attn_fwd_window(qd, kd, vd, 1, window, n_sink)
    sees = torch.zeros(S, dtype=torch.bool)
    sees[at:at + window] = True
    assert torch.isnan(out[:, sees]).all() and torch.isnan(lse[:, :, sees]).all()
    assert_close(out[:, ~sees], want[:, ~sees.numpy()], dtype, "out")
    assert_close(lse[:, :, ~sees], want_l[:, :, ~sees.numpy()], dtype, "lse")
