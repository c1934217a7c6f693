"""GPU tests of how many bits attend_tree keeps of a weight: all 24, in every form of the call.

The first test makes a result of what the two leading bf16 parts of one weight leave of it.  A key
at a distance, of weight w in [1/2, 1), has value 1; two keys in the query's place, of weight 1, have
the values -half and -rest, half = bf16(w), rest = bf16(w - half); every other value is 0.  The sum is
w - half - rest, up to 2^-18, and all sums on the way are multiples of 2^-24 below 1 in size,
which float32 holds.  What may be off: w itself by e = the roundings that tests/cache_util.py counts
for it, up to 12 joins by half a step each (sums of several warps or blocks, softmax factors), the
stored value by half a step.  A weight rounded to two parts gives 0, three times the bound away.
"""
import numpy as np
import pytest
import torch

import oracle
from order_retrieval_gb300 import ZetaCache
from order_retrieval_gb300 import workloads as W

from cache_util import EPS, attend_row, window
from draft_util import Drafting, line

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

GAMMA = 0.5


def _bf16(x):
    return torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).double().item()


def _weight(weight, d, g2=GAMMA ** 2):
    d2 = float((d.astype(np.float64) ** 2).sum())
    return (1 / (1 + d2 / g2) if weight == "cauchy" else np.exp(-d2 / g2)), d2


def _far(weight, d_K, rng):
    """(offset, w, half, rest) of a key whose third part is next to the largest there is."""
    while True:
        d = rng.uniform(0.05, 0.3, d_K).astype(np.float32) / np.float32(np.sqrt(d_K))
        w, _ = _weight(weight, d)
        half = _bf16(w)
        rest = _bf16(w - half)
        if 0.5 <= w < 1 and abs(w - half - rest) >= 0.85 * 2.0 ** -18:
            return d, w, half, rest


@pytest.mark.parametrize("weight", ["cauchy", "softmax"])
@pytest.mark.parametrize("d_K,d_V", [(3, 64), (3, 40), (3, 128), (3, 72), (2, 64), (3, 33), (3, 256),
                                     (5, 64)])
@pytest.mark.parametrize("n", [3, 12, 40])
@pytest.mark.parametrize("where", ["few", "steps", "window", "line"])
def test_a_weight_has_all_its_bits(where, n, d_K, d_V, weight):
    """Both keys among few tokens of the chunk, among whole steps of them, in a window, in a line."""
    rng = np.random.default_rng(n + d_V)
    H, C, k, page = 2, (8 if where == "window" else 64), 8, (8 if where == "window" else 64)
    start = {"few": 5, "steps": 50, "window": 8, "line": 0}[where]
    if where == "window":
        n = min(n, C)
    cache = ZetaCache.empty(8, page, H, d_K, d_V, 64, C, k, 6, torch.bfloat16, weight)
    d, w, half, rest = _far(weight, d_K, rng)
    scale = np.ldexp(np.where(np.arange(d_V) % 3 == 1, -1.0, 1.0), -(np.arange(d_V) % 5))
    at = {"few": (3, 1), "steps": (2, 20), "window": (6, 1), "line": (0, 1)}[where]
    keys = rng.uniform(-0.9, 0.9, (1, H, max(start, 1), d_K)).astype(np.float32)
    vals = np.zeros((1, H, max(start, 1), d_V))
    nk, nv = np.zeros((1, H, n, d_K), np.float32), np.zeros((1, H, n, d_V))
    nv[:] = -rest * scale
    first = 0                                        # the first node that sees all three
    parent = np.full((1, n), -1)
    if where == "line":
        nk[:, :, 0], nv[:, :, 0] = d, scale
        nv[:, :, 1] = -half * scale
        parent[0, 1], parent[0, 2:], first = 0, 1, 2
    else:
        keys[:, :, at[0]], vals[:, :, at[0]] = d, scale
        keys[:, :, at[1]], vals[:, :, at[1]] = 0, -half * scale
    up = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(t).cuda()  # noqa: E731
    bf, f32 = torch.bfloat16, torch.float32
    table = Drafting.ints([np.arange(8) if page == 8 else [5]])
    if start:
        cache.append(up(keys, f32), up(vals, bf), Drafting.ints([0]), Drafting.ints([start]), table)
        cache.order(Drafting.ints([0]), Drafting.ints([start]), table, n=start)
    out, rs = torch.empty(1, H, n, d_V, dtype=bf, device="cuda"), torch.empty(1, H, n, device="cuda")
    cache.attend_tree(torch.zeros(1, H, n, d_K, device="cuda"), up(nk, f32), up(nv, bf),
                      torch.full((H,), GAMMA, device="cuda"), Drafting.ints([start]),
                      Drafting.ints([n]), Drafting.ints(parent), table, out, rs)
    assert int(cache.status.item()) == 0
    if weight == "cauchy":
        e = (d_K + 9) * EPS
    else:
        x = -np.log(w)
        e = (x * (d_K + 5) + 2 * (2 + 1.2 * x) + 2) * EPS
    for h in range(H):
        # every other key's weight is in the sum of weights alone
        total = 2 + w
        if where != "line":
            total += sum(_weight(weight, keys[0, h, j])[0] for j in range(start) if j not in at)
        want = (w - half - rest) * scale / total
        bound = (e * w + 12 * EPS) * np.abs(scale) / total + np.abs(want) * (2.0 ** -8 + 64 * EPS)
        got = out[0, h, first:].double().cpu().numpy()
        assert (np.abs(got - want) <= bound).all(), (got[0, 0], want[0], bound[0])
        assert (bound * 2 < np.abs(want)).all()


class Whole(Drafting):
    """A draft whose plain form allows no rounding of a weight to fewer bits."""

    def plain(self, b, t, h, gone=()):
        w, s = self.w, self.starts[b]
        nodes = line(self.parents[b], t)
        i = s + len(nodes) - 1
        keys = np.concatenate([self.g["k"][b, h, :s], self.kn[b, h, nodes]])
        vals = np.concatenate([self.values[b][h][:s], self.vn[b, h, nodes]])
        q = self.qn[b, h, t]
        win = window(oracle.encode(q[None], w.bits)[0], self.codes[b][h], i, w.C, w.k)
        return (win, *attend_row(q, keys, vals, float(self.g["gamma"][h]), win, i, w.C,
                                 self.weight, 0.0, 2.0 ** -8 if w.v_dtype == "bf16" else EPS))


@pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
@pytest.mark.parametrize("kw", [dict(), dict(d_V=128), dict(d_V=24, d_K=2, bits=21), dict(d_V=250),
                                dict(d_K=5, bits=12), dict(d_V=33, v_dtype="f32"),
                                dict(d_K=8, bits=8, d_V=256)],
                         ids=lambda x: "-".join(f"{a}{b}" for a, b in x.items()) or "base")
def test_every_form_within_float32(kw, weight):
    """All weights in both kernels, in chunks that start on and off whole steps."""
    w = W.Workload(**{**dict(name="draft", B=4, H=2, N=480, d_K=3, d_V=64, k=20, C=120, bits=10,
                             v_dtype="bf16", gamma=(0.4, 1.0), dist="clusters", v_dist="normal",
                             seed=29), **kw})
    d = Whole(w, 32, [200, 480 - 7, 50, 300], [30, 7, 33, 1], 33, weight, kind="bushy")
    d.attend()
    d.check()
