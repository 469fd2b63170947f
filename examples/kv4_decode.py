"""Block decoding over a 4-bit KV cache, end to end on synthetic data.

Every step of a small LLaDA-shaped layer refreshes the rows of its drifting
clusters (the Polestar step), stores them in the 4-bit cache, attends with the
current block's queries, and adds up the weight that the cache's slots draw.
After the last step the cache is cut to half by that weight and attended again.

    python examples/kv4_decode.py [--steps 4] [--keep 0.5]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from drift_aware_kv_spherical_gb300 import workloads as wl   # noqa: E402
from drift_aware_kv_spherical_gb300.pipeline import Pipeline  # noqa: E402

W = wl.Workload("kv4_example", 90, B=2, N=768, d=1024, Hq=8, Hkv=8, dh=128, C=32, iters=4, k=8,
                P=32, V=4096, dtype="bf16", planted=32, noise=1.0, drift_frac=0.05, drift_std=0.5,
                blk_start=512, logit_std=2.0, wq_std=0.02, desc="small LLaDA-shaped layer")


def main(steps=4, keep=0.5):
    """Runs the example; returns (cosine of the outputs before and after the
    eviction, share of the drawn weight that was kept)."""
    dev = "cuda"
    L = wl.make_layer(W, 0, dev)
    H = L["H"]
    pipe = Pipeline(W, layers=1, kv4=True, kmul=2.0 ** -4, vmul=2.0 ** -4)
    kv = pipe.kv4[0]
    O = torch.empty(W.B, W.P, W.Hq, W.dh, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(W.B, W.P, W.Hq, device=dev)
    blk = slice(W.blk_start, W.blk_start + W.P)
    full = (torch.tensor([0, W.N], dtype=torch.int32, device=dev)
            .expand(W.B, W.P, 2).contiguous())
    for t in range(steps):
        if t:
            H = wl.drift_rows(W, H, t)
        Q = wl.make_queries(W, H, L["Wq"])
        st = pipe.state[0]
        if t == 0:      # the window is built: clustered from scratch, every row refreshed
            pipe.layer_step(0, H, Q, L["Wk"], L["Wv"], wl.make_uniforms(W, 0, dev), first=True,
                            full=True)
        else:
            pipe.layer_step(0, H, Q, L["Wk"], L["Wv"])
        pipe.t += 1
        q = Q[:, blk].contiguous()
        kv.attend(q, O, lse, span=full)
        kv.weigh(q, lse, span=full)
        print(f"step {t}: refreshed {int(st.npos.sum()) if t else W.B * W.N} rows, "
              f"lse {float(lse.mean()):.3f}")
    before, drawn = O.float().clone(), kv.w.sum()
    kv.evict(int(W.N * keep), sink=4, recent=W.N - W.blk_start)
    kv.attend(q, O, lse, span=full)
    cos = torch.nn.functional.cosine_similarity(before.flatten(), O.float().flatten(), dim=0)
    share = float(kv.w[:, :, :int(W.N * keep)].sum() / drawn)
    print(f"cut to {int(kv.len[0])} of {W.N} slots: {share:.1%} of the drawn weight kept, "
          f"outputs' cosine {float(cos):.4f}")
    return float(cos), share


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--keep", type=float, default=0.5)
    a = ap.parse_args()
    main(a.steps, a.keep)
