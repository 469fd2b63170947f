"""Queries of a block as a slice of a window's, for layers with and without rotary
positions."""
import numpy as np
import pytest
import torch

import test_gpu_attn as base
import test_gpu_block_attend as block
from drift_aware_kv_spherical_gb300 import polestar as ps
from drift_aware_kv_spherical_gb300 import workloads as wl
from drift_aware_kv_spherical_gb300.pipeline import Pipeline

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_slice_of_the_windows_queries(dtype):
    w = block.LOADS[dtype]
    L, u, logits = block._layer(w)
    pipe = Pipeline(w, layers=1)
    Q = wl.make_queries(w, L["H"], L["Wq"])
    pipe.decode_step(block.FIRST, [L["H"]], [Q], [L["Wk"]], [L["Wv"]], logits, [u])
    T = w.P
    q = Q[:, w.blk_start:w.blk_start + T]
    O, lse = torch.zeros(w.B, T, w.Hq, w.dh, dtype=Q.dtype, device="cuda"), \
        torch.zeros(w.B, T, w.Hq, device="cuda")
    was = Q.clone()
    pipe.attend(0, q, O, lse)
    rows = lambda x: x.reshape(-1, *x.shape[2:])  # noqa: E731
    st = pipe.state[0]
    base._near(rows(O), rows(lse), rows(q), rows(st.Kc), rows(st.Vc), np.arange(w.B + 1) * T,
               np.arange(w.B) * w.N, np.full(w.B, w.N))
    assert torch.equal(Q, was)
    again = torch.zeros_like(O)
    pipe.attend(0, q.contiguous(), again)
    assert torch.equal(O, again)
    with pytest.raises(ValueError, match="one stride"):
        pipe.attend(0, q, torch.zeros_like(Q)[:, :T])
