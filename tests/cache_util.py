"""Plain 64-bit forms of the paged-cache calls and the error bounds the kernels
are held to; numpy only, one (b, h) slice at a time."""
import numpy as np

import oracle

EPS = 2.0 ** -24                       # half a step of float32, relative


def window(q_codes, k_codes, i, C, k):
    """Tokens of position i's window, [] in chunk 0: the k entries around its rank
    among the keys of the chunks before its own, ordered by (code, token)."""
    m = i // C * C
    if m == 0:
        return np.empty(0, np.int64)
    order = np.argsort(k_codes[:m], kind="stable")
    r = int((k_codes[:m] <= q_codes).sum())
    st = min(max(r - (k + 1) // 2, 0), m - k)
    return order[st:st + k]


def attend_row(q, keys, v, gamma, win, i, C, weight, half_w, half_out):
    """(out, rowsum, bound of out, bound of rowsum) of the query q at position i.

    The bounds count roundings.  Weight, relative: the squared distance of d terms
    carries (d + 1) EPS; Cauchy adds gamma^2, its reciprocal, one fma and a
    quotient of at most 2 units (4 EPS + 4 EPS); inverse Euclidean takes half the
    distance's error and a reciprocal root of 2 units; the softmax multiplies the
    error of (m - d2) / gamma^2 (d + 5 roundings of d2 and m each) by its size and
    adds an exponential of 2 + 1.2 |x| units.  A weight that enters a matrix
    product is rounded once more (half_w).  Sums of L terms in any order add
    L EPS of their absolute value, joining partial sums and the quotient 16 EPS,
    the stored value half a step (half_out)."""
    j = np.concatenate([win, np.arange(i // C * C, i + 1)])
    d2 = ((q[None].astype(np.float64) - keys[j].astype(np.float64)) ** 2).sum(1)
    d = q.shape[0]
    g2 = float(gamma) ** 2
    if weight == "cauchy":
        w = 1 / (1 + d2 / g2)
        ew = np.full(len(j), (d + 9) * EPS)
    elif weight == "softmax":
        x = (d2 - d2.min()) / g2
        w = np.exp(-x)
        ew = ((d2 + d2.min()) / g2 * (d + 5) + 2 * (2 + 1.2 * x) + 2) * EPS
    else:
        w = 1 / np.sqrt(d2 + 1e-12)
        ew = np.full(len(j), (d + 2 + 4) * EPS)
    s = w.sum()
    a = w / s
    vj = v[j].astype(np.float64)
    out = a @ vj
    size = a @ np.abs(vj)
    mean_e = float(a @ ew)
    sums = (len(j) + 16) * EPS
    b_out = (a * ew) @ np.abs(vj) + size * (mean_e + half_w + 2 * sums) + np.abs(out) * half_out
    return out, s, b_out + 1e-30, s * (mean_e + sums)


class Sequence:
    """One sequence's tokens on the host and what the calls should make of them."""

    def __init__(self, q, k, v, C, ksel, bits, gamma, weight):
        """q, k [H, N, d_K] float32, v [H, N, d_V] float64, gamma [H]."""
        self.q, self.k, self.v, self.C, self.ksel = q, k, v, C, ksel
        self.gamma, self.weight = gamma, weight
        self.qc = np.stack([oracle.encode(x, bits) for x in q])
        self.kc = np.stack([oracle.encode(x, bits) for x in k])

    def prefix(self, h, c):
        """(codes, tokens) of prefix c."""
        m = c * self.C
        order = np.argsort(self.kc[h, :m], kind="stable")
        return self.kc[h, :m][order], order

    def row(self, h, i, half_w, half_out):
        win = window(self.qc[h, i], self.kc[h], i, self.C, self.ksel)
        return (win, *attend_row(self.q[h, i], self.k[h], self.v[h], self.gamma[h], win, i,
                                 self.C, self.weight, half_w, half_out))
