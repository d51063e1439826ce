"""Attention over shared prefixes against plain forms in 64 bits: groups of every kind beside sequences that share nothing,
prefixes that end at tile and page borders, types, head layouts, trees, hints that are wrong, and a run of the calls of
parallel sampling together (fork, reserve, rotary append, shared attention, drawn tokens), captured and replayed."""
import numpy as np
import pytest
import torch

import _paged_plain as paged
import _samples_plain as plain
from _util import cuda, host, status_ok
from test_gpu_paged import Cache, binary, i32

pytestmark = pytest.mark.gpu

EDEVICE = 5


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gb300 as m
    m.lib()
    m.debug_share_from(1)  # small groups too
    yield m
    m.debug_share_from(0)


def share(c, groups):
    """Sequences of one group hold its first member's pages for `slots` slots: groups {(members): slots}."""
    t = host(c.table)
    for members, slots in groups.items():
        lead = members[0]
        for b in members[1:]:
            t[b, :slots] = t[lead, :slots]
            for x in (c.K, c.V):
                x[b][:, :slots * c.P] = x[lead][:, :slots * c.P]
    c.table.copy_(torch.tensor(t))


def run(sdv, c, q, lens, news, group, M, parents=None, ws=None):
    B, H, D = len(lens), q.shape[2], q.shape[3]
    out = torch.full(q.shape, 123.0, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(B, M, H, c.k.shape[1], D)) if ws is None else ws
    sdv.paged_attn_shared(cuda(q), c.pages, c.table, i32(lens), i32(group), out, ws, n_new=i32(news) if news is not None else None,
                          parent=i32(parents) if parents is not None else None)
    return out


def compare(out, c, q, lens, news, parents=None):
    out = host(out)
    for b, (L, n) in enumerate(zip(lens, news)):
        assert np.all(out[b, n:] == 123.0)  # rows behind the last new one are left alone
        if n:
            ref, tol = paged.attention(q[b, :n], c.K[b], c.V[b], paged.seen_rows(L, n, parents[b] if parents is not None else None, 0, 0))
            err = np.abs(out[b, :n] - ref)
            assert np.all(err <= tol), f"sequence {b}: worst {(err / tol).max():.3g} x of the bound"


def check(sdv, seed, lens, news, groups, M, H, H_kv, D, P, dtype, nhd=False, parents=None, group=None, qscale=1.0):
    rng = np.random.default_rng(seed)
    c = Cache(sdv, rng, lens, news, M, H_kv, D, P, dtype, nhd)
    share(c, groups)
    if group is None:
        group = [-1] * len(lens)
        for members in groups:
            for b in members:
                group[b] = members[0]
    q = (rng.standard_normal((len(lens), M, H, D)) * qscale).astype(np.float32)
    out = run(sdv, c, q, lens, news, group, M, parents)
    status_ok()
    compare(out, c, q, lens, news, parents)
    return c, q, out


SIZES = [(128, 16, 2, 8, 1, False), (128, 64, 2, 10, 5, True), (64, 8, 3, 3, 2, True), (64, 32, 1, 7, 16, False),
         (256, 16, 2, 4, 3, False), (256, 128, 1, 8, 4, True), (128, 192, 1, 16, 7, False), (128, 32, 4, 4, 1, True)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("D,P,H_kv,H,M,nhd", SIZES)
def test_groups_beside_each_other(sdv, dtype, D, P, H_kv, H, M, nhd):
    """A group of four, one of two and one whose common part is under a tile, sequences alone (one with a group's number, one
    without rows, one without new rows inside a group), lengths at the borders of tiles and pages."""
    n = -(-640 // P)  # slots of the first group
    lens = [n * P, 10, n * P + 1, 700 + n * P, 0, n * P + 64, 400, 333, 2 * P + 70, 2 * P + 3, n * P + 9, 65]
    news = [M, max(1, M - 1), M, 1, M, M, M, M, M, M, 0, M]
    small = max(1, 63 // P) if P < 64 else 0  # slots under a tile
    groups = {(0, 2, 3, 5): n, (6, 7): 320 // P if P <= 64 else 333 // P, (8, 9): min(2, small)}
    group = [0, -1, 0, 0, -1, 0, 6, 6, 8, 8, 0, 11]
    check(sdv, D + P + M, lens, news, groups, M, H, H_kv, D, P, dtype, nhd, group=group)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("R,M,H,H_kv,D", [(2, 1, 4, 4, 64), (3, 1, 8, 1, 128), (9, 5, 8, 1, 128), (40, 3, 16, 2, 128), (17, 16, 8, 1, 64), (5, 2, 4, 2, 256),
                                         (2, 1, 1, 1, 128), (33, 1, 4, 1, 256)])
def test_query_rows_of_a_group(sdv, dtype, R, M, H, H_kv, D):
    """From two to thousands of query rows over one prefix."""
    lens = [256 + (7 * i) % 90 for i in range(R)]
    news = [M - (i % M) for i in range(R)]
    check(sdv, R, lens, news, {tuple(range(R)): 16}, M, H, H_kv, D, 16, dtype)


@pytest.mark.parametrize("dtype", ["f16", "i8"])
@pytest.mark.parametrize("M", [6, 16])
def test_trees(sdv, dtype, M):
    parents = [binary(M), [-1] + [0] * (M - 1), list(range(-1, M - 1)), [-1] + [max(0, i - 2) for i in range(1, M)]]
    check(sdv, M, [128, 190, 200, 128], [M, M, M - 2, M], {(0, 1, 2): 8}, M, 8, 2, 128, 16, dtype, parents=parents)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
def test_long_prefixes_cut_between_ctas(sdv, dtype):
    lens = [20000, 20100, 20037, 50]
    check(sdv, 1, lens, [1, 2, 3, 3], {(0, 1, 2): 1240}, 3, 4, 1, 128, 16, dtype)


@pytest.mark.parametrize("rows", [63, 64, 65])
def test_the_least_that_is_shared(sdv, rows):
    """Around the number of tiles from which on a prefix is computed once: 3 other members of 2 heads by 5 tiles."""
    try:
        for tiles in (29, 30, 31, 1 << 30):
            sdv.debug_share_from(tiles)
            check(sdv, rows, [256 + rows] * 4, [2] * 4, {(0, 1, 2, 3): (256 + rows) // 8}, 2, 4, 2, 64, 8, "f16")
    finally:
        sdv.debug_share_from(1)


def test_prefixes_that_differ_in_size_by_far(sdv):
    """Rows of large scores in the prefix alone, or behind it alone: the joined softmax is one of them."""
    for qscale in (40.0, 1e-3):
        check(sdv, 2, [256, 300, 640], [2, 2, 2], {(0, 1, 2): 16}, 2, 8, 2, 128, 16, "f16", qscale=qscale)


def test_wrong_hints_change_nothing(sdv):
    """Groups of sequences that share nothing, or in a part only; a member that left; numbers of other sequences."""
    lens, news, P = [300, 310, 320, 330, 200], [2, 1, 2, 2, 2], 16
    for group in ([0, 0, 0, 0, 0], [4, 4, 4, 4, 4], [3, 3, 1, 1, 1], [-1] * 5, [0, 1, 2, 3, 4]):
        check(sdv, 3, lens, news, {(0, 2, 3): 12}, 2, 8, 2, 128, P, "f16", group=group)
    # one member's table differs in the middle of the others' common part
    rng = np.random.default_rng(4)
    c = Cache(sdv, rng, lens, news, 2, 2, 128, P, "f16")
    share(c, {(0, 1, 2, 3): 18})
    own = Cache(sdv, rng, lens, news, 2, 2, 128, P, "f16")  # other values for a page of its own
    page = int(c.order[c.used])
    c.table[1, 9] = page
    for x, vals, src in ((c.k, c.K, own.K), (c.v, c.V, own.V)):
        x[page] = torch.tensor(src[1][:, 144:160]).to(x.dtype).cuda()
        vals[1][:, 144:160] = x[page].double().cpu().numpy()
    q = rng.standard_normal((5, 2, 8, 128)).astype(np.float32)
    for group in ([0] * 5, [0, -1, 0, 0, -1], [1, 1, 2, 2, 2]):
        out = run(sdv, c, q, lens, news, group, 2)
        status_ok()
        compare(out, c, q, lens, news)


def test_bad_groups_lengths_and_pages(sdv):
    lens, news = [100, 140, 200], [2, 2, 2]

    def go(group=(0, 0, 0), lens_=lens, news_=news, spoil=None):
        c = Cache(sdv, np.random.default_rng(5), lens, news, 2, 2, 128, 16, "f16")
        share(c, {(0, 1, 2): 5})
        if spoil is not None:
            c.table[spoil[0], spoil[1]] = spoil[2]
        q = np.random.default_rng(6).standard_normal((3, 2, 4, 128)).astype(np.float32)
        out = run(sdv, c, q, lens_, news_, group, 2)
        torch.cuda.synchronize()
        return c, q, out, sdv.device_status()

    for group in ((3, 0, 0), (-2, 0, 0), (0, 1 << 30, 0)):
        c, q, out, st = go(group)
        assert st == EDEVICE
        compare(out, c, q, lens, news)
    for lens_, news_ in (([-1, 140, 200], news), ([1 << 20, 140, 200], news), (lens, [3, 2, 2]), (lens, [-1, 2, 2])):
        c, q, out, st = go(lens_=lens_, news_=news_)
        assert st == EDEVICE and torch.all(out[0] == 123.0)
        compare(out[1:], type("C", (), dict(K=c.K[1:], V=c.V[1:])), q[1:], lens[1:], news[1:])
    # a page that is missing in one member ends its group's prefix there; the member reads zeros, as in sd_paged_attn
    for page in (-1, 1 << 20):
        c, q, out, st = go(spoil=(1, 2, page))
        assert st == EDEVICE
        compare(torch.stack([out[0], out[2]]), type("C", (), dict(K=[c.K[0], c.K[2]], V=[c.V[0], c.V[2]])), q[[0, 2]], [100, 200], [2, 2])


def test_unseen_rows_may_hold_anything(sdv):
    """NaN in everything behind the sequences' rows and in pages that nobody holds (Cache puts it there), infinities in V of a
    prefix row reach all that see it, in that column alone."""
    c, q, _ = check(sdv, 7, [192, 200, 260], [2, 2, 2], {(0, 1): 12}, 2, 4, 2, 128, 16, "bf16", group=[0, 0, 0])
    c.v[c.table[0, 3], 1, 5, 17] = float("inf")
    out = run(sdv, c, q, [192, 200, 260], [2, 2, 2], [0, 0, -1], 2)
    torch.cuda.synchronize()
    bad = ~np.isfinite(host(out))
    want = np.zeros(bad.shape, bool)
    want[:2, :, 2:, 17] = True
    assert np.array_equal(bad, want)


def test_the_same_bits_again_and_other_sizes_on_one_workspace(sdv):
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(20, 5, 16, 2, 128))
    for seed, (R, M, H, D) in enumerate([(20, 5, 16, 128), (3, 1, 4, 64), (7, 2, 8, 128), (20, 5, 16, 128)]):
        rng = np.random.default_rng(seed)
        lens, news = [320 + 3 * i for i in range(R)], [M] * R
        c = Cache(sdv, rng, lens, news, M, 2, D, 16, "f16")
        share(c, {tuple(range(R)): 20})
        q = rng.standard_normal((R, M, H, D)).astype(np.float32)
        a = run(sdv, c, q, lens, news, [0] * R, M, ws=ws)
        b = run(sdv, c, q, lens, news, [0] * R, M, ws=ws)
        status_ok()
        assert torch.equal(a, b)
        compare(a, c, q, lens, news)


@pytest.mark.parametrize("H,M", [(2, 2), (16, 2)])
def test_as_many_sequences_as_a_call_takes(sdv, H, M):
    """1024 sequences in 512 pairs, and in one group; narrow and wide rows behind the prefix."""
    B, P, D = 1024, 64, 64
    rng = np.random.default_rng(8)
    lens = [64 + b % 7 for b in range(B)]
    pages = 2 * B
    k, v = (torch.randn(pages, 1, P, D, device="cuda", dtype=torch.float16) for _ in range(2))
    for pairs in (True, False):
        t = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2).clone()
        t[:, 0] = t[:, 0] // 4 * 4 if pairs else 0
        group = [b // 2 * 2 if pairs else 5 for b in range(B)]
        q = cuda(rng.standard_normal((B, M, H, D)).astype(np.float32))
        out, ref = torch.zeros_like(q), torch.zeros_like(q)
        pg = sdv.KvPages(k, v)
        sdv.paged_attn_shared(q, pg, t, i32(lens), i32(group), out, sdv.workspace(sdv.paged_attn_shared_workspace_bytes(B, M, H, 1, D)))
        sdv.paged_attn(q, pg, t, i32(lens), ref, sdv.workspace(sdv.paged_attn_workspace_bytes(B, M, H, 1, D)))
        status_ok()
        kk = torch.cat([k[t[:, 0].long()], k[t[:, 1].long()]], 2)[:, 0].double()
        vv = torch.cat([v[t[:, 0].long()], v[t[:, 1].long()]], 2)[:, 0].double()
        s = torch.einsum("bmhd,bnd->bmhn", q.double(), kk) / 8.0
        j, L = torch.arange(128, device="cuda"), i32(lens)
        see = j[None, None, :] <= L[:, None, None] + torch.arange(M, device="cuda")[None, :, None]
        p = torch.softmax(s.masked_fill(~see[:, :, None, :], float("-inf")), -1)
        exact = torch.einsum("bmhn,bnd->bmhd", p, vv)
        # as _paged_plain.attention's bound, with |q| |k| of at most 64 elements
        bound = (2 * ((D + 3) * plain.U * (q.double().abs().amax() * kk.abs().amax() * 64 / 8) + 4 * plain.U) + 8 * (80 + 16) * plain.U) * vv.abs().amax()
        assert torch.all((out - exact).abs() <= bound) and (out - exact).norm() <= 1e-5 * exact.norm()
        assert (ref - exact).norm() <= 1e-5 * exact.norm()


def test_columns_of_wider_rows(sdv):
    """Queries and outputs whose rows are columns of wider tensors; the columns beside them are left alone."""
    rng = np.random.default_rng(9)
    lens, news, M = [128, 150, 129], [2, 1, 2], 2
    c = Cache(sdv, rng, lens, news, M, 2, 128, 16, "f16")
    share(c, {(0, 1, 2): 8})
    wide = rng.standard_normal((3, M, 7, 128)).astype(np.float32)
    to = torch.full((3, M, 9, 128), 123.0, device="cuda")
    sdv.paged_attn_shared(cuda(wide)[:, :, 2:6], c.pages, c.table, i32(lens), i32([0, 0, 0]), to[:, :, 1:5],
                          sdv.workspace(sdv.paged_attn_shared_workspace_bytes(3, M, 4, 2, 128)), n_new=i32(news))
    status_ok()
    compare(to[:, :, 1:5].contiguous(), c, wide[:, :, 2:6], lens, news)
    assert torch.all(to[:, :, 0] == 123.0) and torch.all(to[:, :, 5:] == 123.0)


def test_two_streams_at_once(sdv):
    """Calls beside each other, each with its own workspace."""
    rng = np.random.default_rng(11)
    sets = []
    for D in (128, 64):
        lens, news = [640, 700, 650, 30], [2, 2, 1, 2]
        c = Cache(sdv, rng, lens, news, 2, 2, D, 16, "f16")
        share(c, {(0, 1, 2): 40})
        q = rng.standard_normal((4, 2, 8, D)).astype(np.float32)
        sets.append((c, q, lens, news, torch.cuda.Stream(), sdv.workspace(sdv.paged_attn_shared_workspace_bytes(4, 2, 8, 2, D))))
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(10):
        for i, (c, q, lens, news, s, ws) in enumerate(sets):
            with torch.cuda.stream(s):
                outs[i] = run(sdv, c, q, lens, news, [0] * 4, 2, ws=ws)
    torch.cuda.synchronize()
    status_ok()
    for out, (c, q, lens, news, _, _) in zip(outs, sets):
        compare(out, c, q, lens, news)


def test_parallel_sampling(sdv):
    """One prompt forked into six samples: reserve, rotary append, shared attention, a head, drawn tokens and commit, as one
    captured graph replayed for 40 steps; every step's rows, outputs and tokens against plain forms, the prompt's pages still
    shared at the end."""
    rng = np.random.default_rng(10)
    B, H, H_kv, D, P, V, L0 = 6, 4, 2, 64, 16, 500, 200
    hid = H * D
    n_pages = 200
    k, v = (torch.zeros(n_pages, H_kv, P, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pg, rope = sdv.KvPages(k, v), sdv.Rope(D, base=500000.0, scaling="yarn", factor=4.0, original=128, low=1.0, high=32.0)
    freq = np.array(rope.inv_freq)
    width = 20
    refs, table, lens = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), torch.full((B, width), -1, dtype=torch.int32, device="cuda"), i32([0] * B)
    missing, pws = i32([0]), sdv.workspace(sdv.pages_workspace_bytes(n_pages, B, width))
    # the prompt, into sequence 0
    embed = rng.standard_normal((V, hid + 2 * H_kv * D)).astype(np.float32)
    head = cuda((rng.standard_normal((hid, V)) * 2).astype(np.float32))
    prompt = rng.integers(0, V, L0)
    first = i32([L0] + [0] * (B - 1))
    sdv.pages_reserve(pg, refs, table, lens, L0, missing, pws, n_new=first)
    line = torch.zeros(B, L0, H + 2 * H_kv, D, device="cuda")
    line[0] = cuda(embed[prompt]).view(L0, -1, D)
    sdv.paged_append_rope(None, line[:, :, H:H + H_kv], line[:, :, H + H_kv:], pg, table, lens, rope, None, n_new=first)
    sdv.paged_commit(pg, table, lens, L0, first)
    sdv.pages_fork(refs, table, lens, P, i32([0] * 5), i32([1, 2, 3, 4, 5]))
    status_ok()
    E, one = cuda(embed), i32([1] * B)
    token, u, q = i32([7] * B), torch.zeros(B, device="cuda"), torch.zeros(B, 1, H, D, device="cuda")
    out, logits = torch.zeros(B, 1, H, D, device="cuda"), torch.zeros(B, V, device="cuda")
    T, top_k, top_p = torch.full((B,), 0.9, device="cuda"), i32([100] * B), torch.full((B,), 0.9, device="cuda")
    rows, group, prob = torch.zeros(B, 1, H + 2 * H_kv, D, device="cuda"), i32([0] * B), torch.zeros(B, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(B, 1, H, H_kv, D))

    def step():
        sdv.pages_reserve(pg, refs, table, lens, 1, missing, pws)
        torch.index_select(E, 0, token, out=rows.view(B, -1))
        sdv.paged_append_rope(rows[:, :, :H], rows[:, :, H:H + H_kv], rows[:, :, H + H_kv:], pg, table, lens, rope, q)
        sdv.paged_attn_shared(q, pg, table, lens, group, out, ws)
        torch.matmul(out.view(B, -1), head, out=logits)
        sdv.sample(logits, u, token, temperature=T, top_k=top_k, top_p=top_p, prob=prob)
        sdv.paged_commit(pg, table, lens, 1, one)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.matmul(out.view(B, -1), head, out=logits)  # (the library's own start, outside the capture)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        text = [list(prompt) for _ in range(B)]
        for _ in range(40):
            was = host(token)
            u.copy_(cuda(rng.random(B).astype(np.float32) * 0.999))
            graph.replay()
            s.synchronize()
            got, lo, tab = host(out), host(logits), host(table)
            for b in range(B):
                text[b].append(int(was[b]))
                n = len(text[b])
                x = embed[text[b]].reshape(n, H + 2 * H_kv, D)
                kk, _ = plain.turn(x[:, H:H + H_kv], np.arange(n), freq, rope.scale, False)
                qq, _ = plain.turn(x[-1:, :H], [n - 1], freq, rope.scale, False)
                pages, at = tab[b, np.arange(n) // P], np.arange(n) % P
                held = host(k)[pages, :, at].astype(np.float64)
                assert np.all(np.abs(held - kk) <= 2.0 ** -10 * np.abs(kk) + 1e-5)
                ref, tol = paged.attention(qq.astype(np.float32), held.transpose(1, 0, 2), host(v)[pages, :, at].astype(np.float64).transpose(1, 0, 2),
                                           np.ones((1, n), bool))
                # (the queries are off by 9 u of |a| + |b| each, a score by as much of sum |q k| / sqrt(D))
                extra = 2 * 18 * plain.U * np.abs(qq).max() * np.abs(held).max() * D / np.sqrt(D) * np.abs(host(v)).max()
                assert np.all(np.abs(got[b] - ref) <= tol + extra)
                plain.check_row(lo[b], float(u[b]), float(np.float32(0.9)), 100, float(np.float32(0.9)), 0.0, int(token[b]), float(prob[b]), None)
    status_ok()
    tab = host(table)
    assert host(lens).tolist() == [L0 + 40] * B and int(missing) == 0
    assert np.all(tab[:, :L0 // P] == tab[0, :L0 // P]) and len(set(tab[:, L0 // P])) == B
