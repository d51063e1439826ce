"""Plain forms of the calls on a cache in pages, in 64 bits and one row at a time (numpy, host)."""
import numpy as np

U = 2.0 ** -24


def path_of(parent, i):
    got = []
    while i >= 0:
        got.append(i)
        i = int(parent[i]) if parent is not None else i - 1
    return sorted(got)


def seen_rows(L, n, parent, window, sinks):
    """[n][L + n] bool: what each new row sees.  Path node k stands at position L + k."""
    see = np.zeros((n, L + n), bool)
    for i in range(n):
        path = path_of(parent, i)
        at = L + len(path) - 1
        j = np.arange(L)
        see[i, :L] = True if not window else (j > at - window) | (j < sinks)
        for k, t in enumerate(path):
            see[i, L + t] = not window or L + k > at - window or L + k < sinks
    return see


def attention(q, K, V, see):
    """q [n][H][D], K / V [H_kv][rows][D] and see [n][rows] -> (out, tol) [n][H][D] in 64 bits.

    tol bounds the kernel's fp32 arithmetic: a score is off by at most (D + 3) u sum|q_d k_d| / sqrt(D) (operands
    split to 2^-22 = 4 u or better, fp32 sums, 2 u for the scaling and 1 u for an 8-bit row's scale) and 4 u for
    exp2f, so a weight by 2 delta relative (numerator and sum); weights, products and sums over NK rows and the
    joins add 8 (NK + 16) u, all relative to sum_j P_j |v_j|."""
    n, H, D = q.shape
    g = H // K.shape[0]
    out, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    for h in range(H):
        for i in range(n):
            j = np.nonzero(see[i])[0]
            if not len(j):
                continue
            k, v = K[h // g, j].astype(np.float64), V[h // g, j].astype(np.float64)
            s = k @ q[i, h].astype(np.float64) / np.sqrt(D)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ v
            delta = (D + 3) * U * (np.abs(k) @ np.abs(q[i, h]).astype(np.float64)).max() / np.sqrt(D) + 4 * U
            tol[i, h] = (2 * delta + 8 * (len(j) + 16) * U) * (p @ np.abs(v)) + 1e-30
    return out, tol


def codes(x):
    """8-bit codes and scale of rows [.., D] in the fp32 arithmetic that the calls name."""
    x = x.astype(np.float32)
    scale = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = (x / scale[..., None]).astype(np.float32)
    whole = np.trunc(y)
    whole = whole + np.where(np.abs(y - whole) >= 0.5, np.sign(y), 0)
    return np.where(scale[..., None] > 0, np.clip(whole, -127, 127), 0).astype(np.int8), scale


class Pool:
    """Counts, tables and lengths, with the calls' rules one entry at a time."""

    def __init__(self, n_pages, B, width, P):
        self.refs, self.P = [0] * n_pages, P
        self.table, self.lens = [[-1] * width for _ in range(B)], [0] * B

    def fork(self, pairs):
        dsts = [d for _, d in pairs]
        srcs = {s for s, _ in pairs}
        for s, d in pairs:
            if dsts.count(d) > 1 or d in srcs:
                continue
            self.free([(d, 0)])
            self.lens[d] = self.lens[s]
            for x in range(-(-self.lens[s] // self.P)):
                if self.table[s][x] >= 0:
                    self.table[d][x] = self.table[s][x]
                    self.refs[self.table[s][x]] += 1

    def free(self, which):
        for b, keep in which:
            for x in range(-(-keep // self.P), len(self.table[b])):
                if self.table[b][x] >= 0:
                    self.refs[self.table[b][x]] -= 1
                    self.table[b][x] = -1
            self.lens[b] = min(self.lens[b], keep)

    def trim(self, window, sinks):
        for b, L in enumerate(self.lens):
            for x, pg in enumerate(self.table[b]):
                if pg >= 0 and x * self.P >= sinks and (x + 1) * self.P <= L - window + 1:
                    self.refs[pg] -= 1
                    self.table[b][x] = -1

    def reserve(self, n_new):
        """Returns (missing, copies [(from, to, rows)])."""
        refs, table, copies = list(self.refs), [list(t) for t in self.table], []
        free = [p for p, r in enumerate(refs) if r == 0]
        short = 0
        for b, n in enumerate(n_new):
            for x in range(self.lens[b] // self.P, -(-(self.lens[b] + n) // self.P) if n else 0):
                was = table[b][x]
                if was >= 0 and refs[was] == 1:
                    continue
                if not free:
                    short += 1
                    if was >= 0:
                        refs[was] -= 1
                    continue
                to = free.pop(0)
                refs[to] = 1
                table[b][x] = to
                if was >= 0:
                    refs[was] -= 1
                    rows = max(0, min(self.P, self.lens[b] - x * self.P))
                    if rows:
                        copies.append((was, to, rows))
        if short:
            return short, []
        self.refs, self.table = refs, table
        return 0, copies

    def compact(self):
        """Returns (n_live, remap, moves)."""
        n_live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n_live) if self.refs[p] == 0]
        remap = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        moves = []
        for p in range(n_live, len(self.refs)):
            if self.refs[p]:
                to = holes.pop(0)
                remap[p] = to
                self.refs[to], self.refs[p] = self.refs[p], 0
                moves.append((p, to))
        self.table = [[remap[e] if e >= 0 else e for e in t] for t in self.table]
        return n_live, remap, moves
