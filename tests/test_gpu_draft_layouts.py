"""GPU tests of attend_tree's tile kernel in every layout its rule may choose: one or two groups of 8
nodes to a block, 1, 2, 4 or 8 blocks to them."""
import numpy as np
import pytest
import torch

from order_retrieval_gb300 import workloads as W

from draft_util import Drafting


def layout(S, n, C, d_V):
    """The rule of tile_layout (cache_tree.cu): (groups, blocks) for S slices of n nodes."""
    groups = 2 if d_V <= 64 and (n > 8 or S <= 64) else 1
    rows, warps, blocks = 8 * groups, 4 * groups, 1
    tiles = S * -(-n // rows)
    while (blocks < 8 and tiles * blocks * 2 <= 152 * (4 // groups)
           and (min(n, rows) > warps * blocks or C > 256 * blocks)):
        blocks *= 2
    return groups, blocks


# (B, H, n, C, d_V): layout
CASES = {
    (10, 4, 20, 256, 64): (2, 2), (30, 8, 20, 256, 64): (2, 1), (4, 4, 5, 256, 64): (2, 1),
    (3, 4, 20, 512, 64): (2, 2), (3, 4, 20, 1024, 64): (2, 4), (10, 5, 11, 1024, 40): (2, 4),
    (2, 4, 20, 2048, 64): (2, 8), (4, 8, 16, 2048, 64): (2, 8), (5, 8, 16, 2048, 32): (2, 4),
    (1, 1, 3, 2048, 64): (2, 8),
    (10, 8, 8, 256, 64): (1, 2), (50, 8, 8, 256, 64): (1, 1), (10, 8, 4, 256, 64): (1, 1),
    (10, 8, 5, 1024, 64): (1, 4), (9, 8, 8, 2048, 64): (1, 8), (20, 8, 6, 2048, 64): (1, 2),
    (2, 4, 4, 256, 128): (1, 1), (3, 4, 20, 512, 128): (1, 2), (3, 4, 20, 1024, 72): (1, 4),
    (2, 4, 20, 2048, 128): (1, 8), (25, 8, 20, 1024, 96): (1, 1),
}


def test_the_cases_reach_every_layout():
    assert {(g, b) for g in (1, 2) for b in (1, 2, 4, 8)} == set(CASES.values())
    for (B, H, n, C, d_V), want in CASES.items():
        assert layout(B * H, n, C, d_V) == want, (B, H, n, C, d_V)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("v_dtype,weight", [("bf16", "cauchy"), ("bf16", "softmax"),
                                            ("f32", "softmax")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_every_layout(case, v_dtype, weight):
    """Chunks that are full, half full, empty: blocks with many of the shared keys, few and none."""
    B, H, n, C, d_V = case
    w = W.Workload(name="draft", B=B, H=H, N=2 * C, d_K=3, d_V=d_V, k=20, C=C, bits=10,
                   v_dtype=v_dtype, gamma=(0.4, 1.0), dist="uniform", v_dist="normal", seed=37)
    rng = np.random.default_rng(B + n)
    starts = rng.integers(0, w.N, B)
    starts[:4] = [C + C // 2, C, 2 * C - n // 2 - 1, C + 17][:B]
    counts = np.maximum(1, rng.integers(n // 2, n + 1, B))
    counts[0] = n
    d = Drafting(w, 64, starts, counts, n, weight, kind="bushy")
    d.attend()
    picks = {(int(b), int(t)) for b in rng.integers(0, B, 5) for t in rng.integers(0, n, 3)}
    d.check(picks | {(0, 0), (0, n - 1), (B - 1, 0), (min(2, B - 1), 0)}, heads=(0, H - 1))
