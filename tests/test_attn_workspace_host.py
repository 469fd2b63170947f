"""How much workspace attention over packed sequences asks for, without a GPU."""
import itertools
import os

import pytest


@pytest.fixture(scope="module")
def ps():
    from drift_aware_kv_spherical_gb300 import _build, polestar
    if not os.path.exists(polestar.LIB_PATH):
        _build.build()
    polestar.Library.load()
    return polestar


def test_partial_sums_are_those_of_the_rows_that_run_side_by_side(ps):
    """Shares are made until some 600 CTAs of up to 16 rows (152 of up to 256) have one
    each, so their sums of dh + 2 floats are no more than 152 * 256 * 258 * 4 bytes, 40 MB,
    and twice that where a batch runs two kernels."""
    most = 0
    for S, (Hq, Hkv), dh, q, k in itertools.product(
            (1, 2, 3, 17, 200, 5000), ((1, 1), (28, 4), (32, 8), (32, 32), (64, 1)), (64, 128, 256),
            (1, 5, 9, 300, 4096, 16384), (1, 700, 5000, 32768, 65536, 1 << 20)):
        for Tq in sorted({S, q, q + S - 1, S * q}):
            if Tq * Hq <= 1 << 30:
                for max_q in {q, Tq}:
                    n = ps.ps_workspace_bytes(ps.OP_ATTN, B=S, N=k, Hq=Hq, Hkv=Hkv, dh=dh, P=Tq,
                                              k=max_q)
                    assert n <= 80 << 20, (S, Hq, Hkv, dh, Tq, max_q, k, n)
                    most = max(most, n)
    assert most > 1 << 20


def test_a_token_beside_a_long_prompt(ps):
    size = lambda **k: ps.ps_workspace_bytes(ps.OP_ATTN, **k)  # noqa: E731
    # S * 8 rows a KV head in at most 512 shares
    assert size(B=2, N=32768, Hq=28, Hkv=4, dh=128, P=4097, k=4096) <= 2 * 8 * 4 * 76 * 130 * 4 + 512
    assert size(B=2, N=65536, Hq=32, Hkv=8, dh=128, P=16385, k=16384) <= 2 * 8 * 8 * 38 * 130 * 4 + 512
