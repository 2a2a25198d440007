"""Whether a cut or a draw is the one that the definition gives for a sum within
1e-11 of itself of the true one: no row is left out, however near its border lies.
Sums have 64 bits of mantissa or more; nothing here shares code with the kernels."""
import numpy as np

NEAR = 1e-11  # of the sum: what the interface names


class Row:
    """A row of logits with its weights, and what of it top-k leaves."""

    def __init__(self, z, T=1.0, k=0):
        assert np.finfo(np.longdouble).nmant >= 63
        self.z, self.T, self.k = np.asarray(z, np.float64), float(np.float32(T)), k or len(z)
        self.order = np.argsort(-self.z, kind="stable")
        self.w = np.exp((self.z - self.z.max()).astype(np.longdouble) / np.longdouble(self.T))
        self.total = np.cumsum(self.w[self.order[:self.k]])  # of the k first, descending

    def count_of(self, kept):
        """How many are kept, which have to be the order's first."""
        n = int(kept.sum())
        assert kept[self.order[:n]].all()
        return n

    def check_count(self, n, p):
        """The n first are the fewest that reach p of the k's sum."""
        S, goal = self.total[-1], np.longdouble(np.float32(p)) * self.total[-1]
        assert 1 <= n <= self.k
        over, under = (self.total[n - 1] - goal) / S, (goal - (self.total[n - 2] if n > 1 else 0)) / S
        assert over >= -NEAR, f"{float(over):.3g} of the sum lack"
        assert n == 1 or under > -NEAR, f"the last is not needed, by {-float(under):.3g} of the sum"

    def check_token(self, token, u, n=None):
        """The token with which, by index, more than u of the n first's sum is reached."""
        at = np.sort(self.order[:self.k if n is None else n])
        sums = np.cumsum(self.w[at])
        j = int(np.searchsorted(at, token))
        assert j < len(at) and at[j] == token, "not of what is kept"
        target = np.longdouble(np.float32(u))
        before, upto = (sums[j - 1] if j else 0) / sums[-1], sums[j] / sums[-1]
        assert before <= target + NEAR, f"too far, by {float(before - target):.3g} of the sum"
        assert upto > target - NEAR, f"not far enough, by {float(target - upto):.3g} of the sum"

    def near(self, edges, lo, hi, least, most, how_many):
        """Floats between lo and hi that lie between `least` and `most` of the sum from
        one of the edges (shares of it), on either side."""
        edges = edges[(edges > lo) & (edges < hi)]
        f = edges.astype(np.float32)
        out = []
        for g in (np.nextafter(f, np.float32(0)), f, np.nextafter(f, np.float32(1))):
            gap = np.abs(g.astype(np.longdouble) - edges)
            out.append(g[(gap >= least) & (gap <= most)])
        out = np.unique(np.concatenate(out))
        return out[np.linspace(0, len(out) - 1, min(how_many, len(out))).astype(int)] if len(out) else out

    def near_draws(self, how_many, least=1.5 * NEAR, most=2e-10, n=None):
        at = np.sort(self.order[:self.k if n is None else n])
        sums = np.cumsum(self.w[at])
        return self.near(sums / sums[-1], 0.05, 0.95, least, most, how_many)

    def near_cuts(self, how_many, least=1.5 * NEAR, most=2e-10, lo=0.3, hi=0.9999):
        return self.near(self.total / self.total[-1], lo, hi, least, most, how_many)
