"""The README's calls on packed sequences, run as they stand there."""
import os

import numpy as np
import pytest
import torch

import test_gpu_attn as base
from drift_aware_kv_spherical_gb300 import polestar as ps

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.mark.parametrize("B,T,N,Hq,Hkv", [(4, 32, 768, 32, 32), (8, 1, 4096, 28, 4)])
def test_calls_on_packed_sequences(B, T, N, Hq, Hkv):
    blocks = open(README).read().split("```python\n")[1:]
    code, = [b.split("```")[0] for b in blocks if "ps.OP_ATTN" in b]
    g = torch.Generator().manual_seed(B)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    R, V = B * T, 1000
    x = dict(ps=ps, B=B, T=T, N=N, Hq=Hq, Hkv=Hkv, Q=bf(B, T, Hq, 128), K=bf(B, T, Hkv, 128),
             V=bf(B, T, Hkv, 128), Qr=bf(B, T, Hq, 128), Kc=bf(B, N, Hkv, 128),
             Vc=bf(B, N, Hkv, 128), O=bf(R, Hq, 128), q_off=torch.arange(B + 1, **i32) * T,
             k_off=torch.arange(B, **i32) * N, lengths=torch.arange(B, **i32) * 7 + N // 2,
             logits=bf(R, V), u=torch.rand(R, dtype=torch.float64, device="cuda"),
             token=torch.full((R,), -9, **i32), prob=torch.zeros(R, device="cuda"),
             t=torch.full((R,), 0.8, device="cuda"), k=torch.full((R,), 50, **i32),
             p=torch.full((R,), 0.9, device="cuda"))
    exec(code, x)
    torch.cuda.synchronize()
    ps.ps_check()
    lse = torch.zeros(R, Hq, device="cuda")
    rows = lambda n: x[n].view(-1, *x[n].shape[2:])  # noqa: E731
    a = (np.arange(B + 1) * T, np.arange(B) * N, x["lengths"].cpu().numpy() + T)
    ps.ps_attn(rows("Qr"), rows("Kc"), rows("Vc"), torch.empty_like(x["O"]), lse, q_off=x["q_off"],
               k_off=x["k_off"], k_len=x["lengths"] + T, causal=True, max_q=T, max_k=N, ws=x["ws"])
    base._near(x["O"], lse, rows("Qr"), rows("Kc"), rows("Vc"), *a, causal=True)
    assert ((x["token"] >= 0) & (x["token"] < V) & (x["prob"] > 0)).all()
