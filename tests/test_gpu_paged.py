"""The calls on a cache in pages against plain forms in 64 bits: attention over ragged batches, types, head layouts,
page sizes, trees, windows and what stands in unseen rows; appended rows and codes bit for bit; page plans, copies
and tables entry for entry; a run of cycles of them together, captured into a graph and replayed."""
import numpy as np
import pytest
import torch

import _paged_plain as plain
from _util import cuda, host, status_ok

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
EDEVICE = 5


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gb300 as m
    m.lib()
    return m


def i32(v):
    return torch.tensor(np.asarray(v, np.int32)).cuda()


class Cache:
    """A pool with rows placed through shuffled tables; everything that no sequence holds is NaN (8-bit: NaN scales)."""

    def __init__(self, sdv, rng, lens, news, M, H_kv, D, P, dtype, nhd=False, spare=3, hold=None, scale=1.0):
        self.sdv, self.P, self.dtype = sdv, P, dtype
        B = len(lens)
        width = max(1, max(-(-(L + M) // P) for L in lens)) + 1
        n_pages = sum(-(-(L + n) // P) for L, n in zip(lens, news)) + spare
        order = rng.permutation(n_pages)
        table = np.full((B, width), -1, np.int32)
        at = 0
        self.K, self.V = [], []  # the rows' values per sequence, [H_kv][rows][D] in 64 bits
        shape = (n_pages, P, H_kv, D) if nhd else (n_pages, H_kv, P, D)
        fill = torch.full if dtype == "i8" else (lambda s, v, **k: torch.full(s, float("nan"), **k))
        k, v = (fill(shape, 77, dtype=TYPES[dtype]) for _ in range(2))
        k, v = (x.permute(0, 2, 1, 3) if nhd else x for x in (k, v))
        ks, vs = (torch.full((n_pages, H_kv, P), float("nan")) for _ in range(2))
        for b, (L, n) in enumerate(zip(lens, news)):
            rows = L + n
            vals = []
            for t, s in ((k, ks), (v, vs)):
                x = rng.standard_normal((H_kv, rows, D)).astype(np.float32) * (scale if t is k else 1.0)
                if dtype == "i8":
                    c, sc = plain.codes(x)
                    # row scales of very different sizes, some 0
                    sc = (sc * np.exp2(rng.integers(-12, 3, sc.shape))).astype(np.float32) if t is v else sc
                    sc[rng.random(sc.shape) < 0.02] = 0.0
                    x = torch.tensor(c)
                    vals.append(c.astype(np.float64) * sc[..., None])
                else:
                    x = torch.tensor(x).to(TYPES[dtype])
                    vals.append(x.double().numpy())
                for slot in range(-(-rows // P)):
                    lo, hi = slot * P, min(rows, (slot + 1) * P)
                    if t is k:
                        table[b, slot] = order[at + slot]
                    pg = int(table[b, slot])
                    t[pg, :, :hi - lo] = x[:, lo:hi]
                    if dtype == "i8":
                        s[pg, :, :hi - lo] = torch.tensor(sc[:, lo:hi])
            at += -(-rows // P)
            self.K.append(vals[0])
            self.V.append(vals[1])
        self.order, self.used = order, at
        stride = (lambda t: t.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)) if nhd else (lambda t: t.contiguous().cuda())
        self.k, self.v = stride(k), stride(v)
        self.ks, self.vs = (ks.cuda(), vs.cuda()) if dtype == "i8" else (None, None)
        self.table = torch.tensor(table).cuda()
        self.pages = sdv.KvPages(self.k, self.v, self.ks, self.vs)

    def rows(self, b, lo, hi):
        """Rows [lo, hi) of sequence b as the pool holds them: K, V [H_kv][hi-lo][D] in 64 bits."""
        j = torch.arange(lo, hi)
        pg, r = self.table[b].cpu()[j // self.P].long(), j % self.P
        got = []
        for t, s in ((self.k, self.ks), (self.v, self.vs)):
            x = t.cpu()[pg, :, r].double()
            got.append((x * s.cpu()[pg, :, r].double()[..., None] if s is not None else x).permute(1, 0, 2).numpy())
        return got


def binary(M):
    return [-1] + [(i - 1) // 2 for i in range(1, M)]


def run_attn(sdv, cache, q, lens, news, M, parents, window, sinks):
    B, H, D = len(lens), q.shape[2], q.shape[3]
    out = torch.full(q.shape, 123.0, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_workspace_bytes(B, M, H, cache.k.shape[1], D))
    sdv.paged_attn(cuda(q), cache.pages, cache.table, i32(lens), out, ws, n_new=i32(news),
                   parent=i32(parents) if parents is not None else None, window=window, sinks=sinks)
    torch.cuda.synchronize()
    status_ok()
    return host(out)


def check_attn(sdv, seed, lens, news, M, H, H_kv, D, P, dtype, nhd=False, parents=None, window=0, sinks=0, scale=1.0, qscale=1.0):
    rng = np.random.default_rng(seed)
    c = Cache(sdv, rng, lens, news, M, H_kv, D, P, dtype, nhd, scale=scale)
    q = (rng.standard_normal((len(lens), M, H, D)) * qscale).astype(np.float32)
    out = run_attn(sdv, c, q, lens, news, M, parents, window, sinks)
    for b, (L, n) in enumerate(zip(lens, news)):
        assert np.all(out[b, n:] == 123.0)  # rows behind the last new one are left alone
        if n == 0:
            continue
        see = plain.seen_rows(L, n, parents[b] if parents is not None else None, window, sinks)
        ref, tol = plain.attention(q[b, :n], c.K[b], c.V[b], see)
        err = np.abs(out[b, :n] - ref)
        assert np.all(err <= tol), f"sequence {b}: worst {(err / tol).max():.3g} x of the bound"


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("D,P,H_kv,H,M,nhd", [
    (128, 16, 2, 8, 1, False), (128, 64, 2, 10, 5, True), (64, 8, 3, 3, 2, True), (64, 32, 1, 7, 16, False),
    (256, 16, 2, 4, 3, False), (256, 128, 1, 8, 4, True), (128, 192, 1, 16, 7, False), (128, 32, 4, 4, 1, True),
])
def test_ragged_batches(sdv, dtype, D, P, H_kv, H, M, nhd):
    """Lengths from 0 over tile and page borders to some hundreds, new rows from none to M."""
    lens = [0, 1, P - 1, P, 63, 64, 65, 129, 500, 777]
    news = [M, max(1, M - 1), M, 0, 1, M, M, max(1, M // 2), M, M]
    check_attn(sdv, D + P + M, lens, news, M, H, H_kv, D, P, dtype, nhd)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("H,M", [(8, 6), (32, 16)])
def test_trees(sdv, dtype, H, M):
    lens, news = [0, 60, 64, 700], [M, M, M - 2, M]
    parents = [binary(M), [-1] + [0] * (M - 1), list(range(-1, M - 1)), [-1] + [max(0, i - 2) for i in range(1, M)]]
    check_attn(sdv, 5, lens, news, M, H, 4, 128, 16, dtype, parents=parents)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (17, 4), (64, 0), (100, 5), (128, 64), (300, 70), (5000, 3), (33, 10000)])
@pytest.mark.parametrize("tree", [False, True])
def test_windows_and_sinks(sdv, dtype, window, sinks, tree):
    M = 5
    lens, news = [0, 3, 64, 130, 400, 1000], [5, 5, 4, 5, 1, 5]
    check_attn(sdv, window, lens, news, M, 4, 2, 64, 16, dtype, parents=[binary(M)] * len(lens) if tree else None, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("M,H,H_kv,D", [(3, 3, 1, 128), (3, 3, 1, 64), (4, 8, 2, 64), (4, 5, 1, 256), (16, 8, 1, 256), (5, 10, 2, 64), (11, 3, 1, 128), (16, 4, 1, 64), (13, 10, 2, 128), (16, 8, 1, 64),
                                        (9, 15, 1, 128), (16, 40, 1, 64), (16, 64, 1, 128)])
def test_many_rows_per_kv_head(sdv, dtype, M, H, H_kv, D):
    """From 9 to 1024 query rows of a KV head, some sequences with fewer, contexts over tile and CTA borders."""
    lens, news = [0, 62, 64, 130, 1500], [M, 1, M - 1, 0, M]
    check_attn(sdv, M * H, lens, news, M, H, H_kv, D, 16, dtype)
    check_attn(sdv, M * H + 1, [400, 90], [M, M], M, H, H_kv, D, 32, dtype, nhd=True, parents=[binary(M)] * 2, window=100, sinks=3)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("H", [1, 4])
def test_many_rows_over_long_contexts(sdv, dtype, H):
    """Runs of more tiles than any ring holds, cut between CTAs."""
    check_attn(sdv, 77, [30011, 5000], [16, 9], 16, H * 4, 1, 128, 64, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
def test_long_contexts_are_split_and_joined(sdv, dtype):
    check_attn(sdv, 9, [20011, 0, 64, 9000], [3, 1, 3, 2], 3, 4, 1, 128, 64, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
def test_sharp_scores(sdv, dtype):
    check_attn(sdv, 11, [700, 64], [2, 2], 2, 4, 2, 128, 16, dtype, scale=6.0, qscale=6.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tiny_and_huge_queries(sdv, dtype):
    check_attn(sdv, 12, [300], [2], 2, 2, 1, 128, 16, dtype, scale=1.0, qscale=1e-30)
    check_attn(sdv, 13, [300], [2], 2, 2, 1, 128, 16, dtype, scale=1e-3, qscale=3e3)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_of_many_sequences(sdv, dtype, D):
    """More sequences than the many-row kernel's schedule holds, and as many as it does."""
    rng = np.random.default_rng(D)
    for B in (513, 512):
        lens = rng.integers(0, 150, B).tolist()
        news = rng.integers(0, 4, B).tolist()
        c = Cache(sdv, rng, lens, news, 3, 1, D, 16, dtype)
        q = rng.standard_normal((B, 3, 5, D)).astype(np.float32)
        out = run_attn(sdv, c, q, lens, news, 3, None, 40, 3)
        for b in rng.permutation(B)[:60].tolist():
            if news[b]:
                ref, tol = plain.attention(q[b, :news[b]], c.K[b], c.V[b], plain.seen_rows(lens[b], news[b], None, 40, 3))
                assert np.all(np.abs(out[b, :news[b]] - ref) <= tol)
            assert np.all(out[b, news[b]:] == 123.0)


@pytest.mark.parametrize("dtype,D,B", [("f16", 128, 1024), ("bf16", 64, 1023), ("i8", 128, 700)])
def test_trees_of_more_sequences_than_one_launch_takes(sdv, dtype, D, B):
    """Every argument of the second launch: its tables, lengths, numbers of new rows, trees, strided queries and outputs."""
    rng = np.random.default_rng(B)
    M, H = 7, 3
    lens, news = rng.integers(0, 90, B).tolist(), rng.integers(0, M + 1, B).tolist()
    c = Cache(sdv, rng, lens, news, M, 1, D, 8, dtype)
    parents = [[-1] + [int(rng.integers(0, i)) for i in range(1, M)] for _ in range(B)]
    wide = torch.randn(B, M + 1, 2 * H, D, device="cuda")
    q, outs = wide[:, :M, H:], torch.full((B, M + 2, H, D), 123.0, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_workspace_bytes(B, M, H, 1, D))
    sdv.paged_attn(q, c.pages, c.table, i32(lens), outs[:, 1:M + 1], ws, n_new=i32(news), parent=i32(parents), window=30, sinks=2)
    status_ok()
    assert torch.all(outs[:, 0] == 123.0) and torch.all(outs[:, M + 1] == 123.0)
    out = host(outs)[:, 1:M + 1]
    for b in rng.permutation(B)[:80].tolist() + [0, (B + 1) // 2 - 1, (B + 1) // 2, B - 1]:
        if news[b]:
            ref, tol = plain.attention(host(q[b, :news[b]]), c.K[b], c.V[b], plain.seen_rows(lens[b], news[b], parents[b], 30, 2))
            assert np.all(np.abs(out[b, :news[b]] - ref) <= tol), b
        assert np.all(out[b, news[b]:] == 123.0)


def test_many_sequences(sdv):
    """As many as a call takes."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, 1024).tolist()
    check_attn(sdv, 21, lens, [1 + i % 2 for i in range(1024)], 2, 2, 1, 64, 16, "f16")
    with pytest.raises(sdv.SdError):
        check_attn(sdv, 22, [1] * 1025, [1] * 1025, 1, 1, 1, 64, 16, "f16")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("H", [1, 2, 7, 15, 30])
def test_unseen_rows_may_hold_anything(sdv, dtype, what, H):
    """A tree's sibling and a row behind one position's window hold NaN or infinities in K and V: the positions that do not
    see them are exact, the others are not numbers (or infinite) where V is."""
    rng = np.random.default_rng(4)
    L, M, window, parent = 100, 5, 40, [-1, 0, 0, 1, 2]
    c = Cache(sdv, rng, [L], [M], M, 1, 128, 16, dtype)
    q = rng.standard_normal((1, M, H, 128)).astype(np.float32)
    see = plain.seen_rows(L, M, parent, window, 4)
    bad_old, bad_new = L - window + 1, L + 4  # the first only the root sees, the second only node 4
    assert see[:, bad_old].tolist() == [True, False, False, False, False] and see[:, bad_new].tolist() == [False] * 4 + [True]
    for j in (bad_old, bad_new):
        pg, r = int(c.table[0, j // 16]), j % 16
        for t, s in ((c.k, c.ks), (c.v, c.vs)):
            if dtype == "i8":
                s[pg, :, r] = float(what)
            else:
                t[pg, :, r, 5:70] = float(what)
    out = run_attn(sdv, c, q, [L], [M], M, [parent], window, 4)[0]
    ref, tol = plain.attention(q[0, 1:4], c.K[0], c.V[0], see[1:4])
    assert np.all(np.abs(out[1:4] - ref) <= tol)
    assert not np.isfinite(out[[0, 4]]).all(axis=(1, 2)).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H", [1, 3, 10, 25])
def test_infinite_values_reach_the_rows_that_see_them_alone(sdv, dtype, H):
    """V alone holds an infinity in one column of a new row: the same column of the positions that see it, and nothing else."""
    rng = np.random.default_rng(14)
    L, M = 30, 4
    c = Cache(sdv, rng, [L], [M], M, 1, 64, 8, dtype)
    q = rng.standard_normal((1, M, H, 64)).astype(np.float32)
    j = L + 2
    c.v[int(c.table[0, j // 8]), 0, j % 8, 11] = float("inf")
    out = run_attn(sdv, c, q, [L], [M], M, None, 0, 0)[0]
    see = plain.seen_rows(L, M, None, 0, 0)
    V = c.V[0].copy()
    V[0, j, 11] = 0.0
    ref, tol = plain.attention(q[0], c.K[0], V, see)
    assert np.all(np.isposinf(out[2:, :, 11]))
    out[2:, :, 11] = ref[2:, :, 11]
    assert np.all(np.abs(out - ref) <= tol)


@pytest.mark.parametrize("value", [1e4, 1e10, 1e30, 1e38])
@pytest.mark.parametrize("M,H,D", [(5, 1, 128), (5, 2, 128), (5, 7, 128), (5, 15, 128), (5, 30, 128), (1, 1, 64), (5, 3, 64), (5, 5, 64), (1, 2, 256), (5, 3, 256)])
def test_large_scales_of_unseen_rows(sdv, value, M, H, D):
    """int8 rows whose scales are finite and large where a position does not look: unwritten rows and pages, rows behind the
    window in its first tile (whole tiles come after it), a tree's sibling, a row that the first position alone sees.  The
    positions that do not see them keep the bound of every other case; those that see one (whose K is as it was) too, but for
    what the split leaves: weights times scales in two fp16 parts, in units of U 2^-14 where U is at most twice the largest
    scale that the position sees, are off by half of fp16's least step, 2^-25 of that: 2^-38 of the largest scale seen, times the
    code, for each row (the softmax sum is at least 1 in the same units)."""
    rng = np.random.default_rng(D + H)
    lens, window, sinks, parent = [100, 1000, 70], 40 if M > 1 else 600, 4, [-1, 0, 0, 1, 2][:M]
    c = Cache(sdv, rng, lens, [M] * 3, M, 1, D, 16, "i8")
    q = rng.standard_normal((3, M, H, D)).astype(np.float32)
    for s in (c.ks, c.vs):
        s[torch.isnan(s)] = value
    for b, L in enumerate(lens):
        see = plain.seen_rows(L, M, parent, window, sinks)
        for j in np.nonzero(~see.all(0))[0].tolist():
            pg, r = int(c.table[b, j // 16]), j % 16
            if not see[:, j].any():
                c.ks[pg, :, r] = c.vs[pg, :, r] = value
            elif j in (L - window + 1, L + 4):
                c.vs[pg, :, r] = value
                c.V[b][:, j] = c.v[pg, :, r].cpu().double().numpy() * float(c.vs[pg, 0, r])
    out = run_attn(sdv, c, q, lens, [M] * 3, M, [parent] * 3, window, sinks)
    for b, L in enumerate(lens):
        see = plain.seen_rows(L, M, parent, window, sinks)
        ref, tol = plain.attention(q[b], c.K[b], c.V[b], see)
        j = torch.arange(L + M)
        pg, r = c.table[b].cpu()[j // 16].long(), j % 16
        code, scale = c.v.cpu()[pg, 0, r].double().numpy(), c.vs.cpu()[pg, 0, r].double().numpy()
        for i in range(M):
            if np.abs(c.V[b][0, see[i]]).max() < 1e37:  # (else the output is past fp32's range)
                left = 2.0 ** -38 * scale[see[i]].max() * np.abs(code[see[i]]).sum(0)
                assert np.all(np.abs(out[b, i] - ref[i]) <= tol[i] + left), (b, i)


@pytest.mark.parametrize("value", [1e4, 1e10, 1e30])
@pytest.mark.parametrize("M,H,D", [(5, 1, 128), (5, 2, 128), (5, 7, 128), (5, 15, 128), (16, 16, 128), (5, 3, 64), (5, 5, 64), (16, 8, 64), (2, 2, 256), (5, 3, 256)])
def test_large_scales_ahead_of_whole_tiles(sdv, value, M, H, D):
    """The first rows of the window and of the sinks, which the first positions alone see, have large V scales, and tiles that every
    position sees come after them, some with zeros for scales: each position keeps its bound (that of the split, where it sees
    one: 2^-38 of the largest scale seen, as above)."""
    rng = np.random.default_rng(D + H)
    lens, window, sinks, parent = [1000, 700, 650, 610], 600, 5, binary(M)
    c = Cache(sdv, rng, lens, [M] * 4, M, 1, D, 16, "i8")
    q = rng.standard_normal((4, M, H, D)).astype(np.float32)

    def at(b, j):
        return int(c.table[b, j // 16]), j % 16

    for b, L in enumerate(lens):
        see = plain.seen_rows(L, M, parent, window, sinks)
        for j in range(L - window - 30, L - window + 2):
            if j >= sinks and not see[:, j].all():
                c.vs[at(b, j)[0], :, at(b, j)[1]] = value
        if b == 1:  # whole tiles of zeros behind the window's first
            for j in range(L - window + 60, L - window + 200):
                c.vs[at(b, j)[0], :, at(b, j)[1]] = 0.0
        c.V[b] = c.rows(b, 0, L + M)[1]
    out = run_attn(sdv, c, q, lens, [M] * 4, M, [parent] * 4, window, sinks)
    for b, L in enumerate(lens):
        see = plain.seen_rows(L, M, parent, window, sinks)
        ref, tol = plain.attention(q[b], c.K[b], c.V[b], see)
        j = torch.arange(L + M)
        pg, r = c.table[b].cpu()[j // 16].long(), j % 16
        code, scale = c.v.cpu()[pg, 0, r].double().numpy(), c.vs.cpu()[pg, 0, r].double().numpy()
        for i in range(M):
            left = 2.0 ** -38 * scale[see[i]].max() * np.abs(code[see[i]]).sum(0)
            assert np.all(np.abs(out[b, i] - ref[i]) <= tol[i] + left), (b, i)


@pytest.mark.parametrize("power", [-100, -60, -20, 20, 60, 100])
@pytest.mark.parametrize("M,H,D,window", [(3, 1, 128, 0), (3, 4, 128, 0), (5, 10, 128, 300), (5, 30, 64, 300), (5, 2, 64, 70), (3, 4, 256, 300)])
def test_scales_of_any_size(sdv, power, M, H, D, window):
    """int8 rows whose V scales are all near a power of two far from 1: the outputs are that much larger or smaller."""
    rng = np.random.default_rng(D + H)
    lens = [700, 64, 130]
    c = Cache(sdv, rng, lens, [M] * 3, M, 1, D, 16, "i8")
    q = rng.standard_normal((3, M, H, D)).astype(np.float32)
    c.vs *= 2.0 ** power
    out = run_attn(sdv, c, q, lens, [M] * 3, M, [binary(M)] * 3, window, 3)
    for b, L in enumerate(lens):
        ref, tol = plain.attention(q[b], c.K[b], c.V[b], plain.seen_rows(L, M, binary(M), window, 3))
        assert np.all(np.abs(out[b] * 2.0 ** -power - ref) <= tol), b


@pytest.mark.parametrize("M,H,D", [(2, 2, 128), (2, 8, 128), (5, 8, 128), (16, 8, 128), (5, 5, 64), (2, 4, 256)])
def test_rows_whose_values_are_zero(sdv, M, H, D):
    """int8 rows with a V scale of 0: all from row 32 on (half a tile and whole ones), all of a sequence, and the new rows alone."""
    rng = np.random.default_rng(29)
    lens = [40, 700, 50, 100]
    c = Cache(sdv, rng, lens, [M] * 4, M, 1, D, 16, "i8")
    for b, lo in ((0, 32), (1, 32), (2, 0), (3, 100)):
        j = torch.arange(lo, lens[b] + M)
        c.vs[c.table[b].cpu()[j // 16].long(), :, j % 16] = 0.0
        c.V[b][:, lo:] = 0.0
    q = rng.standard_normal((4, M, H, D)).astype(np.float32)
    out = run_attn(sdv, c, q, lens, [M] * 4, M, None, 0, 0)
    for b, L in enumerate(lens):
        ref, tol = plain.attention(q[b], c.K[b], c.V[b], plain.seen_rows(L, M, None, 0, 0))
        assert np.all(np.abs(out[b] - ref) <= tol), b


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H", [1, 3, 8])
def test_cut_tiles_in_a_row_that_hold_no_numbers(sdv, dtype, H):
    """Four tiles one after the other of which each position sees a part, all with rows of NaN where it does not look: behind the
    first rows and the window, siblings, rows past the end.  The same call many times."""
    rng = np.random.default_rng(30)
    L, M, window, sinks, parent = 1000, 16, 70, 40, binary(16)
    c = Cache(sdv, rng, [L] * 3, [M] * 3, M, 1, 128, 16, dtype)
    see = plain.seen_rows(L, M, parent, window, sinks)
    for b in range(3):
        j = torch.tensor(np.nonzero(~see.any(0))[0])
        c.k[c.table[b].cpu()[j // 16].long(), :, j % 16] = float("nan")
        c.v[c.table[b].cpu()[j // 16].long(), :, j % 16] = float("nan")
        c.v[int(c.table[b, (L + M - 1) // 16]), :, (L + M - 1) % 16, 3] = float("inf")  # the last row: a sibling of the others
    q = cuda(rng.standard_normal((3, M, H, 128)).astype(np.float32))
    ws = sdv.workspace(sdv.paged_attn_workspace_bytes(3, M, H, 1, 128))
    outs = torch.zeros(100, 3, M, H, 128, device="cuda")
    lens, par = i32([L] * 3), i32([parent] * 3)
    for o in outs:
        sdv.paged_attn(q, c.pages, c.table, lens, o, ws, parent=par, window=window, sinks=sinks)
    status_ok()
    assert torch.equal(outs.nan_to_num(7.0), outs[:1].nan_to_num(7.0).expand_as(outs))
    for b in range(3):
        ref, tol = plain.attention(host(q[b]), c.K[b], c.V[b], see)
        assert np.all(np.abs(host(outs[0, b]) - ref)[:-1] <= tol[:-1]), b


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,D", [(1, 64), (1, 128), (3, 128), (10, 64), (10, 128), (25, 128), (1, 256), (3, 256)])
@pytest.mark.parametrize("L,window", [(300, 0), (300, 150), (9000, 0)])
def test_infinite_values_of_committed_rows(sdv, dtype, H, D, L, window):
    """V holds infinities and NaN in rows of tiles that every position sees, and in cut ones: the columns that the formula makes
    infinite or NaN are no numbers (an infinity has the formula's sign), and the others are exact."""
    rng = np.random.default_rng(31)
    M, sinks = 4, 3
    c = Cache(sdv, rng, [L], [M], M, 1, D, 16, dtype)
    q = (rng.standard_normal((1, M, H, D)) * 0.3).astype(np.float32)  # (no weight below fp32's range)
    see = plain.seen_rows(L, M, None, window, sinks)
    V, want = c.V[0].copy(), np.zeros((M, D))
    first = max(0, L - window + 1 if window else 0)
    places = [(first + 70, 5, np.inf), (first + 75, 6, -np.inf), (first + 20, 7, np.inf), (first + 90, 7, -np.inf), (first + 100, 8, np.nan),
              (L + 1, 9, np.inf), (first + 80, 9, np.inf), (L + 2, 10, -np.inf), (first + 71, 10, np.inf), (first + 60, D - 1, np.inf), (L, 63, -np.inf)]
    if window:
        places += [(first, 11, np.inf), (first, 12, np.inf), (first + 90, 12, np.inf), (first - 30, 13, np.inf), (1, 14, -np.inf)]
    for j, d, x in places:
        c.v[int(c.table[0, j // 16]), 0, j % 16, d] = float(x)
        V[0, j, d] = 0.0
        with np.errstate(invalid="ignore"):
            want[see[:, j], d] += x
    out = run_attn(sdv, c, q, [L], [M], M, None, window, sinks)[0]
    ref, tol = plain.attention(q[0], c.K[0], V, see)
    for i in range(M):
        fine = want[i] == 0
        assert np.all(np.abs(out[i][:, fine] - ref[i][:, fine]) <= tol[i][:, fine])
        got = out[i][:, ~fine]
        assert np.all(np.isnan(got) | (got == want[i][~fine])), i


def test_strided_queries_and_outputs(sdv):
    """q and out as columns of wider rows, whose other columns stay as they are."""
    rng = np.random.default_rng(15)
    lens, M, H, D = [70, 9], 3, 4, 64
    c = Cache(sdv, rng, lens, [M, M], M, 2, D, 16, "f16")
    wide = torch.randn(2, M + 1, 3 * H, D, device="cuda")
    q = wide[:, :M, H:2 * H]
    outs = torch.full((2, M, 2 * H, D), 5.0, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_workspace_bytes(2, M, H, 2, D))
    sdv.paged_attn(q, c.pages, c.table, i32(lens), outs[:, :, H:], ws)
    status_ok()
    assert torch.all(outs[:, :, :H] == 5.0)
    for b, L in enumerate(lens):
        ref, tol = plain.attention(host(q[b]), c.K[b], c.V[b], plain.seen_rows(L, M, None, 0, 0))
        assert np.all(np.abs(host(outs[b, :, H:]) - ref) <= tol)


def test_same_result_as_the_contiguous_cache(sdv):
    """One sequence in pages against sd_attn_decode's contiguous cache (both fp32 from the same fp16 rows)."""
    rng = np.random.default_rng(16)
    L, M, H, H_kv, D = 1500, 5, 8, 2, 128
    c = Cache(sdv, rng, [L], [M], M, H_kv, D, 64, "f16")
    q = rng.standard_normal((1, M, H, D)).astype(np.float32)
    out = run_attn(sdv, c, q, [L], [M], M, [binary(M)], 0, 0)[0]
    kc, vc = cuda(c.K[0].astype(np.float16)), cuda(c.V[0].astype(np.float16))
    flat = torch.empty((M, H, D), device="cuda")
    sdv.attn_decode(cuda(q[0]), kc, vc, L, flat, sdv.workspace(sdv.attn_workspace_bytes(M, H, H_kv, D, L)), i32(binary(M)))
    _, tol = plain.attention(q[0], c.K[0], c.V[0], plain.seen_rows(L, M, binary(M), 0, 0))
    assert np.all(np.abs(out - host(flat)) <= 2 * tol)


@pytest.mark.parametrize("H", [6, 40])
def test_results_repeat_and_the_workspace_is_left_ready(sdv, H):
    rng = np.random.default_rng(17)
    lens = [5000, 300, 0, 12000]
    c = Cache(sdv, rng, lens, [2] * 4, 2, 2, 128, 16, "bf16")
    q = cuda(rng.standard_normal((4, 2, H, 128)).astype(np.float32))
    ws = sdv.workspace(sdv.paged_attn_workspace_bytes(4, 2, H, 2, 128))
    outs = []
    for _ in range(4):
        out = torch.zeros_like(q)
        sdv.paged_attn(q, c.pages, c.table, i32(lens), out, ws)
        outs.append(out)
    status_ok()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_bad_entries_are_reported_and_read_as_zeros(sdv):
    rng = np.random.default_rng(18)
    lens = [40, 40, 40]
    c = Cache(sdv, rng, lens, [1] * 3, 1, 1, 64, 16, "f16")
    q = cuda(rng.standard_normal((3, 1, 1, 64)).astype(np.float32))
    c.table[0, 1] = c.k.shape[0]  # past the pool
    c.table[1, 0] = -1            # a visible row's page is missing
    out = torch.zeros_like(q)
    ws = sdv.workspace(sdv.paged_attn_workspace_bytes(3, 1, 1, 1, 64))
    sdv.paged_attn(q, c.pages, c.table, i32(lens), out, ws)
    assert sdv.device_status() == EDEVICE
    assert np.isfinite(host(out)).all()
    ref, tol = plain.attention(host(q[2]), c.K[2], c.V[2], plain.seen_rows(40, 1, None, 0, 0))
    assert np.all(np.abs(host(out[2]) - ref) <= tol)
    for bad in ([40, -1, 40], [40, 10 ** 6, 40]):
        sdv.paged_attn(q, c.pages, c.table, i32(bad), out, ws, window=8)
        assert sdv.device_status() == EDEVICE
    sdv.paged_attn(q, c.pages, c.table, i32(lens), out, ws, n_new=i32([1, 2, -1]), window=8)
    assert sdv.device_status() == EDEVICE
    sdv.paged_attn(q, c.pages, c.table, i32(lens), out, ws, parent=i32([[0], [-1], [-1]]), window=8)
    assert sdv.device_status() == EDEVICE


@pytest.mark.parametrize("H", [2, 8])
@pytest.mark.parametrize("P", [16, 64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30])
def test_missing_pages_of_8_bit_rows_read_as_zeros(sdv, H, P, value):
    """Entries of visible rows that name no page, in tiles that every position sees and in the last one: zeros, whatever the scales
    of the pool's first page are."""
    rng = np.random.default_rng(28)
    lens, M, D = [700, 130, 40], 2, 128
    while True:
        c = Cache(sdv, rng, lens, [M] * 3, M, 1, D, P, "i8")
        if 0 in c.order[c.used:]:
            break  # nobody holds the first page
    c.ks[0] = c.vs[0] = value
    for b, slot, entry in ((0, 1, -1), (0, 2, c.k.shape[0]), (1, 0, -7), (2, 40 // P, -1)):
        c.table[b, slot] = entry
        c.K[b][:, slot * P:(slot + 1) * P] = 0.0
        c.V[b][:, slot * P:(slot + 1) * P] = 0.0
    q = rng.standard_normal((3, M, H, D)).astype(np.float32)
    out = torch.zeros(3, M, H, D, device="cuda")
    sdv.paged_attn(cuda(q), c.pages, c.table, i32(lens), out, sdv.workspace(sdv.paged_attn_workspace_bytes(3, M, H, 1, D)))
    assert sdv.device_status() == EDEVICE
    for b, L in enumerate(lens):
        ref, tol = plain.attention(q[b], c.K[b], c.V[b], plain.seen_rows(L, M, None, 0, 0))
        assert np.all(np.abs(host(out[b]) - ref) <= tol), b


def test_trimmed_pages_are_not_read(sdv):
    """Pages behind the window are released and their entries cleared: the results stay the same."""
    rng = np.random.default_rng(19)
    lens, M, P, window, sinks = [500, 130, 20], 4, 16, 100, 5
    c = Cache(sdv, rng, lens, [M] * 3, M, 2, 64, P, "bf16")
    q = rng.standard_normal((3, M, 2, 64)).astype(np.float32)
    before = run_attn(sdv, c, q, lens, [M] * 3, M, None, window, sinks)
    refs = torch.zeros(c.k.shape[0], dtype=torch.int32, device="cuda")
    held = c.table[c.table >= 0].long()
    refs[held] = 1
    pool = plain.Pool(c.k.shape[0], 3, c.table.shape[1], P)
    pool.refs, pool.table, pool.lens = refs.tolist(), c.table.tolist(), list(lens)
    pool.trim(window, sinks)
    sdv.pages_trim(refs, c.table, i32(lens), P, window, sinks)
    status_ok()
    assert refs.tolist() == pool.refs and c.table.tolist() == pool.table and sum(pool.refs) < len(held)
    for p in (refs == 0).nonzero().view(-1).tolist():
        c.k[p] = float("nan")
        c.v[p] = float("nan")
    assert np.array_equal(before, run_attn(sdv, c, q, lens, [M] * 3, M, None, window, sinks))


def test_offsets_beyond_32_bits(sdv):
    """Pages so far apart that element offsets pass 2^32 (rows written and read there)."""
    stride, P, D = (1 << 32) // 2 + 1024, 16, 64
    big = [torch.empty(2 * stride + 2 * P * D, dtype=torch.float16, device="cuda") for _ in range(2)]
    k, v = (torch.as_strided(t, (3, 2, P, D), (stride, P * D, D, 1)) for t in big)
    pages = sdv.KvPages(k, v)
    rng = np.random.default_rng(20)
    M, lens = 16, i32([0])
    table = i32([[2, 1]])
    new = rng.standard_normal((2, 1, M, 2, D)).astype(np.float32)
    sdv.paged_append(cuda(new[0]), cuda(new[1]), pages, table, lens)
    sdv.paged_commit(pages, table, lens, M, i32([M]))
    more = rng.standard_normal((2, 1, 3, 2, D)).astype(np.float32)
    sdv.paged_append(cuda(more[0]), cuda(more[1]), pages, table, lens)
    q = rng.standard_normal((1, 3, 2, D)).astype(np.float32)
    out = torch.zeros(1, 3, 2, D, device="cuda")
    sdv.paged_attn(cuda(q), pages, table, lens, out, sdv.workspace(sdv.paged_attn_workspace_bytes(1, 3, 2, 2, D)))
    status_ok()
    K, V = (np.concatenate([new[i, 0], more[i, 0]]).astype(np.float16).astype(np.float64).transpose(1, 0, 2) for i in range(2))
    ref, tol = plain.attention(q[0], K, V, plain.seen_rows(M, 3, None, 0, 0))
    assert np.all(np.abs(host(out[0]) - ref) <= tol)
    refs = i32([0, 1, 1])
    ws = sdv.workspace(sdv.pages_workspace_bytes(3, 1, 2))
    remap, n_live = i32([0] * 3), i32([0])
    sdv.pages_compact(pages, refs, table, remap, n_live, ws)
    sdv.paged_attn(cuda(q), pages, table, lens, out, sdv.workspace(sdv.paged_attn_workspace_bytes(1, 3, 2, 2, D)))
    status_ok()
    assert table.tolist() == [[0, 1]] and remap.tolist() == [-1, 1, 0] and n_live.tolist() == [2]
    assert np.all(np.abs(host(out[0]) - ref) <= tol)


# ---------------------------------------------------------------------------------------------------
# appended and committed rows
# ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("M,D,P,H_kv,nhd,fused", [(1, 128, 16, 1, False, False), (5, 64, 8, 3, True, True), (16, 256, 64, 2, False, True), (300, 128, 32, 2, True, False)])
def test_append(sdv, dtype, M, D, P, H_kv, nhd, fused):
    rng = np.random.default_rng(M + D)
    lens, news = [0, 7, P, 3 * P - 1], [M, max(1, M - 1), 0, M]
    c = Cache(sdv, rng, lens, news, M, H_kv, D, P, dtype, nhd)
    before_k, before_v = c.k.clone(), c.v.clone()
    x = (rng.standard_normal((4, M, 3, H_kv, D)) * np.exp2(rng.integers(-20, 8, (4, M, 1, 1, 1)))).astype(np.float32)
    x[0, 0, 1, 0] = 0.0
    if dtype == "i8":
        x[3, 0, 1, 0, :3] = [127.0, 0.5, -1.5]  # halves away from 0 under a scale of 1
        x[3, 0, 1, 0, 3:] = 1.0
    t = cuda(x)
    k_new, v_new = (t[:, :, 1], t[:, :, 2]) if fused else (t[:, :, 1].contiguous(), t[:, :, 2].contiguous())
    sdv.paged_append(k_new, v_new, c.pages, c.table, i32(lens), n_new=i32(news))
    status_ok()
    touched = torch.zeros(c.k.shape[0], P, dtype=torch.bool)
    for b, (L, n) in enumerate(zip(lens, news)):
        for i in range(n):
            pg, r = int(c.table[b, (L + i) // P]), (L + i) % P
            touched[pg, r] = True
            for col, pool, scales in ((1, c.k, c.ks), (2, c.v, c.vs)):
                if dtype == "i8":
                    code, scale = plain.codes(x[b, i, col])
                    assert np.array_equal(host(pool[pg, :, r]), code) and np.array_equal(host(scales[pg, :, r]), scale)
                else:
                    assert torch.equal(pool[pg, :, r].cpu(), torch.tensor(x[b, i, col]).to(TYPES[dtype]))
    keep = ~touched.cuda()[:, None, :, None].expand_as(c.k)
    for was, now in ((before_k, c.k), (before_v, c.v)):
        same = (was == now) | ((was != was) & (now != now))
        assert bool(same[keep].all())  # nothing else is written


def test_append_of_numbers_that_are_none(sdv):
    rng = np.random.default_rng(31)
    c = Cache(sdv, rng, [0], [4], 4, 1, 64, 16, "i8")
    x = rng.standard_normal((1, 4, 1, 64)).astype(np.float32)
    x[0, 0, 0, 3], x[0, 1, 0, 63], x[0, 2, 0, 0] = np.nan, np.inf, -np.inf
    sdv.paged_append(cuda(x), cuda(x), c.pages, c.table, i32([0]))
    status_ok()
    K, V = c.rows(0, 0, 4)
    assert np.isnan(K[0, :3]).all() and np.isnan(V[0, :3]).all() and np.isfinite(K[0, 3]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_of_appended_rows_that_hold_no_numbers(sdv, D):
    """A row with a NaN has that as its scale, one with an infinity alone that, and their codes are 0."""
    rng = np.random.default_rng(34)
    c = Cache(sdv, rng, [0], [5], 5, 2, D, 16, "i8")
    x = rng.standard_normal((1, 5, 2, D)).astype(np.float32)
    x[0, 0, 0, 3], x[0, 1, 0, D - 1], x[0, 2, 0, 0], x[0, 3, 0, 1], x[0, 3, 0, D - 2] = np.nan, np.inf, -np.inf, np.inf, np.nan
    sdv.paged_append(cuda(x), cuda(-x), c.pages, c.table, i32([0]))
    status_ok()
    pg = int(c.table[0, 0])
    for codes, scales, sign in ((c.k, c.ks, 1), (c.v, c.vs, -1)):
        assert np.array_equal(host(scales[pg, 0, :4]), np.array([np.nan, np.inf, np.inf, np.nan], np.float32), equal_nan=True)
        assert not codes[pg, 0, :4].any()
        for i, h in ((4, 0), (0, 1), (1, 1), (2, 1), (3, 1), (4, 1)):
            code, scale = plain.codes(sign * x[0, i, h])
            assert np.array_equal(host(codes[pg, h, i]), code) and float(scales[pg, h, i]) == scale


def test_append_reports_missing_pages_and_skips_them(sdv):
    rng = np.random.default_rng(32)
    c = Cache(sdv, rng, [10, 10], [4, 4], 4, 1, 64, 8, "f16")
    c.table[0, 1] = -1
    before = c.k.clone()
    x = cuda(rng.standard_normal((2, 4, 1, 64)).astype(np.float32))
    sdv.paged_append(x, x, c.pages, c.table, i32([10, 10]), n_new=i32([4, 0]))
    assert sdv.device_status() == EDEVICE
    assert bool(((before == c.k) | (before != before)).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("D,P,H_kv,nhd", [(128, 8, 2, False), (64, 16, 5, True), (256, 64, 1, False)])
def test_commit(sdv, dtype, D, P, H_kv, nhd):
    rng = np.random.default_rng(D)
    M = 16
    lens, news = [0, 5, P - 1, 100, 3], [M] * 5
    c = Cache(sdv, rng, lens, news, M, H_kv, D, P, dtype, nhd)
    paths = [list(range(16)), [0, 2, 5], [15], [0, 1, 3, 7, 15], []]
    path = np.zeros((5, M), np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    L = i32(lens)
    sdv.paged_commit(c.pages, c.table, L, M, i32([len(p) for p in paths]), path=i32(path))
    status_ok()
    assert L.tolist() == [a + len(p) for a, p in zip(lens, paths)]
    for b, p in enumerate(paths):
        for got, was in zip(c.rows(b, 0, lens[b] + M), (c.K[b], c.V[b])):
            want = was.copy()
            want[:, lens[b]:lens[b] + len(p)] = was[:, [lens[b] + t for t in p]]
            assert np.array_equal(got, want)
    sdv.paged_commit(c.pages, c.table, L, M, i32([1, 0, 2, 0, 16]))  # chains: lengths alone
    status_ok()
    assert L.tolist() == [17, 8, P + 2, 105, 19]


def test_commit_refuses_bad_paths_and_counts(sdv):
    rng = np.random.default_rng(33)
    M = 4
    c = Cache(sdv, rng, [10], [M], M, 1, 64, 8, "f16")
    before = c.k.clone()
    for path, count in (([0, 0, 1, 2], 2), ([0, 2, 1, 3], 3), ([0, 1, 2, 4], 4), ([-1, 1, 2, 3], 1), ([0, 1, 2, 3], 5), ([0, 1, 2, 3], -1)):
        L = i32([10])
        sdv.paged_commit(c.pages, c.table, L, M, i32([count]), path=i32([path]))
        assert sdv.device_status() == EDEVICE and L.tolist() == [10]
    assert bool(((before == c.k) | (before != before)).all())


# ---------------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------------

class Both:
    """A pool on the GPU beside the plain one; contents follow the plain plan row by row."""

    def __init__(self, sdv, n_pages, B, width, P, dtype="f16", nhd=False, H_kv=2, D=64, seed=0):
        self.sdv, self.pool, self.P = sdv, plain.Pool(n_pages, B, width, P), P
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        shape = (n_pages, P, H_kv, D) if nhd else (n_pages, H_kv, P, D)
        if dtype == "i8":
            kv = [torch.randint(-127, 128, shape, dtype=torch.int8, generator=g, device="cuda") for _ in range(2)]
            self.scales = [torch.rand(n_pages, H_kv, P, generator=g, device="cuda") for _ in range(2)]
        else:
            kv = [torch.randn(shape, dtype=TYPES[dtype], generator=g, device="cuda") for _ in range(2)]
            self.scales = [None, None]
        self.kv = [t.permute(0, 2, 1, 3) if nhd else t for t in kv]
        self.pages = sdv.KvPages(*self.kv, *self.scales)
        self.refs, self.table = i32([0] * n_pages), i32([[-1] * width] * B)
        self.lens, self.missing = i32([0] * B), i32([7])
        self.remap, self.n_live = i32([9] * n_pages), i32([0])
        self.ws = sdv.workspace(sdv.pages_workspace_bytes(n_pages, B, width))

    def all(self):
        return self.kv + [s for s in self.scales if s is not None]

    def moved(self, want, copies, rows_of):
        for w, now in zip(want, self.all()):
            for a, b, r in copies:
                w[b, :, :r] = w[a, :, :r]
            assert torch.equal(w, now)

    def reserve(self, n_new, M):
        want = [t.clone() for t in self.all()]
        short, copies = self.pool.reserve(n_new)
        self.sdv.pages_reserve(self.pages, self.refs, self.table, self.lens, M, self.missing, self.ws, n_new=i32(n_new))
        status_ok()
        assert self.missing.tolist() == [short]
        self.moved(want, copies, None)
        self.same()
        return short

    def same(self):
        assert self.refs.tolist() == self.pool.refs
        assert self.table.tolist() == self.pool.table
        assert self.lens.tolist() == self.pool.lens

    def grow(self, add):
        self.pool.lens = [a + b for a, b in zip(self.pool.lens, add)]
        self.lens += i32(add)

    def fork(self, pairs):
        self.pool.fork(pairs)
        self.sdv.pages_fork(self.refs, self.table, self.lens, self.P, i32([s for s, _ in pairs]), i32([d for _, d in pairs]))

    def free(self, which, keep=True):
        self.pool.free(which)
        self.sdv.pages_free(self.refs, self.table, self.lens, self.P, i32([b for b, _ in which]), i32([k for _, k in which]) if keep else None)

    def compact(self):
        want = [t.clone() for t in self.all()]
        n_live, remap, moves = self.pool.compact()
        self.sdv.pages_compact(self.pages, self.refs, self.table, self.remap, self.n_live, self.ws)
        status_ok()
        assert self.n_live.tolist() == [n_live] and self.remap.tolist() == remap
        self.moved(want, [(a, b, self.P) for a, b in moves], None)
        self.same()


@pytest.mark.parametrize("dtype,nhd,P,D", [("f16", False, 16, 64), ("bf16", True, 8, 128), ("i8", False, 32, 64), ("i8", True, 64, 256)])
def test_random_runs_of_page_calls(sdv, dtype, nhd, P, D):
    """Reservations, forks, growth, rollbacks, frees, trims and compactions in random order against the plain pool."""
    rng = np.random.default_rng(P)
    B, width = 12, 20
    m = Both(sdv, 90, B, width, P, dtype, nhd, H_kv=3, D=D)
    ran = set()
    for step in range(60):
        do = rng.choice(["reserve", "reserve", "reserve", "fork", "free", "roll", "trim", "compact"])
        if do == "reserve":
            M = int(rng.integers(1, 4 * P))
            n = [int(min(rng.integers(0, M + 1), width * P - L)) if rng.random() < 0.6 else 0 for L in m.pool.lens]
            if m.reserve(n, M) == 0:
                m.grow([int(rng.integers(0, x + 1)) for x in n])
            else:
                ran.add("short")
        elif do == "fork":
            dst = rng.permutation(B)[:4].tolist()
            src = [b for b in range(B) if b not in dst]
            m.fork([(int(rng.choice(src)), d) for d in dst[:int(rng.integers(1, 5))]])
        elif do == "free":
            m.free([(int(b), 0) for b in rng.integers(0, B, 2)], keep=bool(rng.integers(2)))  # now and then one twice
        elif do == "roll":
            m.free([(b, int(rng.integers(0, m.pool.lens[b] + 1))) for b in rng.permutation(B)[:3].tolist()])
        elif do == "trim":
            w, s = int(rng.integers(1, 5 * P)), int(rng.integers(0, 2 * P))
            m.pool.trim(w, s)
            sdv.pages_trim(m.refs, m.table, m.lens, P, w, s)
        else:
            m.compact()
        status_ok()
        m.same()
        ran.add(do)
    assert ran >= {"reserve", "fork", "free", "roll", "trim", "compact"}


def test_shared_pages_are_copied_before_they_are_written(sdv):
    """All holders of a partly filled page write: each but the last gets a copy of the rows so far; one alone gets one too."""
    m = Both(sdv, 40, 6, 4, 16)
    assert m.reserve([20, 0, 0, 0, 0, 0], 20) == 0
    m.grow([20, 0, 0, 0, 0, 0])
    m.fork([(0, 1), (0, 2), (0, 3)])
    assert m.pool.refs[1] == 4
    assert m.reserve([0, 2, 0, 0, 0, 0], 2) == 0       # one of four
    assert m.reserve([5, 0, 1, 16, 0, 0], 16) == 0     # all that are left: the last keeps the page
    assert m.pool.table[3][1] == 1 and m.pool.refs[1] == 1 and m.pool.refs[0] == 4


def test_reserve_takes_all_or_nothing(sdv):
    m = Both(sdv, 5, 3, 8, 8)
    assert m.reserve([17, 8, 9], 17) == 1   # 3 + 1 + 2 pages of 5
    assert m.pool.refs == [0] * 5
    assert m.reserve([17, 8, 8], 17) == 0


def test_planning_over_many_pages(sdv):
    """A pool of several planning rounds, free pages scattered over all of it."""
    rng = np.random.default_rng(8)
    n, B, width, P = 40000, 64, 300, 8
    m = Both(sdv, n, B, width, P, H_kv=1, D=64)
    taken = rng.random(n) < 0.5
    m.pool.refs = taken.astype(int).tolist()
    at = np.nonzero(taken)[0].tolist()
    for b in range(B):  # the taken ones belong to somebody
        for s in range(width - 20):
            if at:
                m.pool.table[b][s] = at.pop()
    for p in at:
        m.pool.refs[p] = 0
    m.pool.lens = [(width - 20) * P - 3] * B
    m.pool.lens = [min(L, P * sum(e >= 0 for e in t)) for L, t in zip(m.pool.lens, m.pool.table)]
    m.refs.copy_(i32(m.pool.refs)), m.table.copy_(i32(m.pool.table)), m.lens.copy_(i32(m.pool.lens))
    assert m.reserve(rng.integers(0, 100, B).tolist(), 100) == 0
    m.compact()


def test_fork_refuses_what_overlaps(sdv):
    m = Both(sdv, 10, 4, 4, 8)
    m.reserve([8, 0, 0, 0], 8)
    m.grow([8, 0, 0, 0])
    for pairs in ([(0, 1), (2, 1)], [(0, 0)], [(0, 1), (1, 2)], [(0, 4)], [(-1, 2)]):
        before = m.refs.tolist(), m.table.tolist()
        sdv.pages_fork(m.refs, m.table, m.lens, 8, i32([s for s, _ in pairs]), i32([d for _, d in pairs]))
        assert sdv.device_status() == EDEVICE
        if pairs != [(0, 1), (1, 2)]:
            assert (m.refs.tolist(), m.table.tolist()) == before


@pytest.mark.parametrize("length", [-1, -2 ** 31, 33, 2 ** 31 - 1])
def test_page_calls_skip_a_length_that_no_table_holds(sdv, length):
    m = Both(sdv, 20, 4, 4, 8)
    m.reserve([20, 10, 8, 0], 20)
    m.grow([20, 10, 8, 0])
    m.fork([(0, 3)])
    status_ok()
    m.same()
    m.lens[1] = length
    before = m.refs.tolist(), m.table.tolist(), m.lens.tolist()
    sdv.pages_fork(m.refs, m.table, m.lens, 8, i32([1]), i32([2]))
    assert sdv.device_status() == EDEVICE and (m.refs.tolist(), m.table.tolist(), m.lens.tolist()) == before
    sdv.pages_free(m.refs, m.table, m.lens, 8, i32([1]), i32([4]))
    assert sdv.device_status() == EDEVICE and (m.refs.tolist(), m.table.tolist(), m.lens.tolist()) == before
    m.pool.lens[1] = 0  # the plain pool skips it, and trims the others
    m.pool.trim(3, 0)
    m.pool.lens[1] = length
    sdv.pages_trim(m.refs, m.table, m.lens, 8, 3)
    assert sdv.device_status() == EDEVICE
    m.same()


def test_a_count_that_is_not_there_is_reported(sdv):
    m = Both(sdv, 10, 2, 4, 8)
    m.table[0, 0] = 3  # a page that nobody counted, and one past the pool
    m.table[0, 1] = 10
    sdv.pages_free(m.refs, m.table, m.lens, 8, i32([0]))
    assert sdv.device_status() == EDEVICE and m.refs.tolist() == [0] * 10 and m.table.tolist() == [[-1] * 4] * 2
    sdv.pages_free(m.refs, m.table, m.lens, 8, i32([2]))
    assert sdv.device_status() == EDEVICE


def test_other_layers_follow(sdv):
    """One plan, the copies made in two layers' pools."""
    m = Both(sdv, 30, 4, 4, 16, seed=1)
    other = Both(sdv, 30, 4, 4, 16, "bf16", True, D=128, seed=2)
    m.reserve([20, 0, 0, 0], 20)
    m.grow([20, 0, 0, 0])
    m.fork([(0, 1), (0, 2)])
    _, copies = plain_copies(m, [3, 3, 3, 0])
    want = [t.clone() for t in other.kv]
    m.reserve([3, 3, 3, 0], 3)
    sdv.pages_copy(other.pages, m.ws)
    status_ok()
    other.moved(want, copies, None)


def test_a_plan_for_a_larger_pool_is_not_followed(sdv):
    """The copies of a pool of 30 pages on one of 3: those within it are made, the others reported, nothing else is touched."""
    m = Both(sdv, 30, 4, 4, 16, seed=1)
    m.reserve([20, 0, 0, 0], 20)
    m.grow([20, 0, 0, 0])
    m.fork([(0, 1), (0, 2)])
    _, copies = plain_copies(m, [3, 3, 3, 0])
    m.reserve([3, 3, 3, 0], 3)
    small = Both(sdv, 3, 4, 4, 16, seed=2)
    want = [t.clone() for t in small.kv]
    sdv.pages_copy(small.pages, m.ws)
    assert sdv.device_status() == EDEVICE
    small.moved(want, [c for c in copies if max(c[:2]) < 3], None)


def plain_copies(m, n_new):
    import copy
    return copy.deepcopy(m.pool).reserve(n_new)


# ---------------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,window,captured", [("f16", 0, False), ("bf16", 48, True), ("i8", 0, True), ("i8", 30, False)])
def test_cycles(sdv, dtype, window, captured):
    """Cycles as a program runs them: pages reserved, a tree's rows appended, attention, the accepted path committed, pages of
    rejected rows given back, pages behind the window released; a fork halfway.  Eager on a side stream, or one captured
    graph replayed with new contents of the same buffers.  Each cycle's attention against the rows kept in 64 bits."""
    rng = np.random.default_rng(41)
    B, M, H, H_kv, D, P, width, n_pages, sinks = 3, 5, 4, 2, 64, 8, 20, 60, 3
    parent = binary(M)
    shape = (n_pages, H_kv, P, D)
    k, v = (torch.full(shape, 3, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(shape[:3], device="cuda") for _ in range(2))
    pages = sdv.KvPages(k, v, ks, vs)
    refs, table, lens, missing = i32([0] * n_pages), i32([[-1] * width] * B), i32([0] * B), i32([0])
    ws, pws = sdv.workspace(sdv.paged_attn_workspace_bytes(B, M, H, H_kv, D)), sdv.workspace(sdv.pages_workspace_bytes(n_pages, B, width))
    new, q = torch.zeros(2, B, M, H_kv, D, device="cuda"), torch.zeros(B, M, H, D, device="cuda")
    out, par = torch.zeros(B, M, H, D, device="cuda"), i32([parent] * B)
    path, count, n_new, seqs = i32([[0] * M] * B), i32([0] * B), i32([0] * B), i32(list(range(B)))

    def cycle():
        sdv.pages_reserve(pages, refs, table, lens, M, missing, pws, n_new=n_new)
        sdv.paged_append(new[0], new[1], pages, table, lens, n_new=n_new)
        sdv.paged_attn(q, pages, table, lens, out, ws, n_new=n_new, parent=par, window=window, sinks=sinks)
        sdv.paged_commit(pages, table, lens, M, count, path=path)
        sdv.pages_free(refs, table, lens, P, seqs, keep=lens)
        if window:
            sdv.pages_trim(refs, table, lens, P, window, sinks)

    side = torch.cuda.Stream()
    graph = None
    kept = [[np.zeros((H_kv, 0, D)) for _ in range(2)] for _ in range(B)]
    for step in range(14):
        if step == 7:  # sequence 2 becomes a copy of sequence 0
            sdv.pages_fork(refs, table, lens, P, i32([0]), i32([2]))
            kept[2] = [x.copy() for x in kept[0]]
        torch.cuda.synchronize()
        x = rng.standard_normal((2, B, M, H_kv, D)).astype(np.float32)
        qs = rng.standard_normal((B, M, H, D)).astype(np.float32)
        news = [int(n) for n in rng.integers(0, M + 1, B)]
        paths = []
        for n in news:  # a root-to-node path among the new rows
            paths.append(plain.path_of(parent, int(rng.integers(0, n))) if n else [])
        pad = np.zeros((B, M), np.int32)
        for b, p in enumerate(paths):
            pad[b, :len(p)] = p
        new.copy_(torch.tensor(x)), q.copy_(torch.tensor(qs)), path.copy_(torch.tensor(pad))
        n_new.copy_(torch.tensor(news)), count.copy_(torch.tensor([len(p) for p in paths]))
        torch.cuda.synchronize()
        if captured:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    cycle()
            graph.replay()
        else:
            with torch.cuda.stream(side):
                cycle()
        torch.cuda.synchronize()
        status_ok()
        assert missing.tolist() == [0]
        got = host(out)
        for b, (n, p) in enumerate(zip(news, paths)):
            rows = []
            for i in range(2):
                y = x[i, b, :n].transpose(1, 0, 2)
                if dtype == "i8":
                    c, s = plain.codes(y)
                    y = c.astype(np.float64) * s[..., None]
                else:
                    y = torch.tensor(y).to(TYPES[dtype]).double().numpy()
                rows.append(np.concatenate([kept[b][i], y], 1))
            L = kept[b][0].shape[1]
            if n:
                ref, tol = plain.attention(qs[b, :n], rows[0], rows[1], plain.seen_rows(L, n, parent, window, sinks))
                assert np.all(np.abs(got[b, :n] - ref) <= tol), (step, b)
            kept[b] = [r[:, list(range(L)) + [L + t for t in p]] for r in rows]
        assert lens.tolist() == [x[0].shape[1] for x in kept]
        counts = np.bincount(host(table)[host(table) >= 0], minlength=n_pages)
        assert np.array_equal(host(refs), counts)


@pytest.mark.parametrize("H", [4, 32])
def test_two_streams_with_their_own_workspaces(sdv, H):
    rng = np.random.default_rng(51)
    lens = [3000, 100]
    c = Cache(sdv, rng, lens, [2, 2], 2, 2, 128, 16, "f16")
    q = [cuda(rng.standard_normal((2, 2, H, 128)).astype(np.float32)) for _ in range(2)]
    L = i32(lens)
    alone = []
    for x in q:
        o = torch.zeros_like(x)
        sdv.paged_attn(x, c.pages, c.table, L, o, sdv.workspace(sdv.paged_attn_workspace_bytes(2, 2, H, 2, 128)))
        alone.append(o)
    outs = [torch.zeros_like(x) for x in q]
    wss = [sdv.workspace(sdv.paged_attn_workspace_bytes(2, 2, H, 2, 128)) for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, o, w in zip(streams, q, outs, wss):
            with torch.cuda.stream(s):
                sdv.paged_attn(x, c.pages, c.table, L, o, w)
    torch.cuda.synchronize()
    status_ok()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])


def test_python_refuses(sdv):
    c = Cache(sdv, np.random.default_rng(61), [10], [1], 1, 2, 64, 16, "f16")
    q = torch.zeros(1, 1, 4, 64, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_workspace_bytes(1, 1, 4, 2, 64))
    lens = i32([10])
    for bad in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(lens=lens.long()), dict(lens=lens.cpu()), dict(table=c.table.long()),
                dict(out=q.new_zeros(1, 1, 2, 64)), dict(n_new=i32([1, 1])), dict(parent=i32([[-1, 0]])), dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))):
        a = dict(q=q, table=c.table, lens=lens, out=torch.zeros_like(q), n_new=None, parent=None)
        a.update(bad)
        with pytest.raises(ValueError):
            sdv.paged_attn(a["q"], c.pages, a["table"], a["lens"], a["out"], ws, n_new=a["n_new"], parent=a["parent"])
    with pytest.raises(ValueError):
        sdv.KvPages(c.k, c.v[:, :1])
    with pytest.raises(ValueError):
        sdv.KvPages(c.k, c.v.clone().transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        sdv.KvPages(c.k.to(torch.int8), c.v.to(torch.int8))
    with pytest.raises(sdv.SdError):
        sdv.KvPages(c.k, c.v) and sdv.paged_attn(q, c.pages, c.table, lens, torch.zeros_like(q), ws[:256])
