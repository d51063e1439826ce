"""Attention over shared prefixes as a step of a running batch: what is shared, and what a replayed step reads."""
import numpy as np
import pytest
import torch

from _util import cuda, host, status_ok
from test_gpu_paged import Cache, i32
from test_gpu_shared import compare, share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gb300 as m
    m.lib()
    m.debug_share_from(1)  # small groups too
    yield m
    m.debug_share_from(0)


# lengths, new rows, groups (members: shared slots of 16 rows)
STEPS = [([640, 700, 650, 30], [2, 1, 2, 2], {(0, 1, 2): 40}),
         ([100, 1000, 1010, 900], [1, 2, 2, 1], {(1, 2, 3): 56}),
         ([320, 330, 500, 510], [2, 2, 1, 2], {(0, 1): 20, (2, 3): 31}),
         ([70, 64, 800, 17], [2, 2, 2, 2], {}),
         ([640, 640, 640, 640], [1, 1, 1, 2], {(0, 1, 2, 3): 40})]


@pytest.mark.parametrize("H,D,dtype", [(2, 128, "f16"), (16, 64, "bf16"), (16, 128, "f16"), (4, 256, "bf16")])
def test_a_replayed_step_reads_what_was_written_before_it(sdv, H, D, dtype):
    """One graph of an append and the attention (few and many query rows), replayed without a pause while lengths, tables, groups, pages
    and queries change under it: the prefixes' tiles, and so the tiles that each sequence skips, are others each time."""
    M, H_kv, P, width, n_pages = 2, 1, 16, 70, 260
    states = []
    for i, (lens, news, groups) in enumerate(STEPS):
        rng = np.random.default_rng(100 + i)
        used = sum(-(-(a + n) // P) for a, n in zip(lens, news))
        c = Cache(sdv, rng, lens, news, M, H_kv, D, P, dtype, spare=n_pages - used)
        share(c, groups)
        group = [next((m[0] for m in groups if b in m), -1) for b in range(4)]
        table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
        table[:, :c.table.shape[1]] = c.table
        q = rng.standard_normal((4, M, H, D)).astype(np.float32)
        new = [torch.zeros(4, M, H_kv, D, device="cuda") for _ in range(2)]
        k, v = c.k.clone(), c.v.clone()
        for b, (L, n) in enumerate(zip(lens, news)):
            for to, pool, x in ((new[0], k, c.K), (new[1], v, c.V)):
                to[b, :n] = torch.tensor(x[b][:, L:L + n].transpose(1, 0, 2)).float().cuda()
                for j in range(L, L + n):  # the step's append brings them
                    pool[int(table[b, j // P]), :, j % P] = 7.0
        states.append((c, q, lens, news, (k, v, table, i32(lens), i32(news), i32(group), cuda(q), *new)))
    fixed = [torch.zeros_like(x) for x in states[0][4]]
    fk, fv, table, lens, n_new, group, q, k_new, v_new = fixed
    pages, out = sdv.KvPages(fk, fv), torch.zeros(4, M, H, D, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(4, M, H, H_kv, D))

    def step():
        sdv.paged_append(k_new, v_new, pages, table, lens, n_new=n_new)
        sdv.paged_attn_shared(q, pages, table, lens, group, out, ws, n_new=n_new)

    s, outs, order = torch.cuda.Stream(), [], [0, 1, 0, 2, 4, 3, 1, 4, 2, 0, 3, 2]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for i in order:
            for to, x in zip(fixed, states[i][4]):
                to.copy_(x)
            out.fill_(123.0)
            graph.replay()
            outs.append(out.clone())
        s.synchronize()
    status_ok()
    for i, o in zip(order, outs):
        c, q_, lens_, news_, _ = states[i]
        compare(o, c, q_, lens_, news_)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H", [2, 16])
def test_rows_whose_scores_are_all_below_the_range(sdv, D, H):
    """Scores that overflow to minus infinity weigh nothing: zeros come out, shared or alone, as from sd_paged_attn.  (4 log2(e) /
    sqrt(D) times -3e38, summed over D, is under -1e40 in its first 16-bit part; what the part leaves, at most 2^-8 of it on either side, adds up to
    less than 2e38.)"""
    P, lens = 16, [200, 230, 300]
    rng = np.random.default_rng(20)
    pages = 16 * 3
    k = torch.full((pages, 1, P, D), -3e38, device="cuda", dtype=torch.bfloat16)
    v = cuda(rng.standard_normal((pages, 1, P, D)).astype(np.float32)).bfloat16()
    table = np.arange(pages, dtype=np.int32).reshape(3, 16)[:, ::-1].copy()
    table = np.concatenate([table, np.full((3, 6), -1, np.int32)], 1)
    table[:, 16:19] = table[:, :3]  # (300 rows take 19 pages)
    table[1, :8] = table[0, :8]
    q = torch.zeros(3, 1, H, D, device="cuda")
    q[:, :, ::2] = 4.0  # the other heads' scores are 0: the mean of the rows
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(3, 1, H, 1, D))
    pg, t = sdv.KvPages(k, v), torch.tensor(table).cuda()
    for group in ([0, 0, -1], [-1, -1, -1]):
        out, ref = torch.full_like(q, 123.0), torch.full_like(q, 123.0)
        sdv.paged_attn_shared(q, pg, t, i32(lens), i32(group), out, ws)
        sdv.paged_attn(q, pg, t, i32(lens), ref, ws)
        status_ok()
        for o in (host(out), host(ref)):
            assert np.all(o[:, :, ::2] == 0.0)
            for b, L in enumerate(lens):
                rows = host(v.double())[table[b, np.arange(L + 1) // P], 0, np.arange(L + 1) % P]
                # each weight is 1 and at most two roundings of u; the sums of up to 301 terms round 19 times in tiles and joins
                tol = (L + 1 + 80) * 2.0 ** -24 * np.abs(rows).mean(0)
                assert np.all(np.abs(o[b, 0, 1::2] - rows.mean(0)) <= tol)


def expected(table, lens, news, group, P, H_kv, n_pages, least):
    """Query rows that a prefix is computed for: of each group's sequences with new rows, the leading slots that name one page in all of
    them, of whole committed pages, in whole 64-row tiles; nothing where all but one member of each group leave out too little."""
    members = {}
    for b, (n, g) in enumerate(zip(news, group)):
        if n > 0 and 0 <= g < len(lens):
            members.setdefault(g, []).append(b)
    less, rows = 0, 0
    for m in members.values():
        if len(m) < 2:
            continue
        slots = min(lens[b] for b in m) // P
        same = 0
        while same < slots and 0 <= table[m[0]][same] < n_pages and all(table[b][same] == table[m[0]][same] for b in m):
            same += 1
        tiles = same * P // 64
        less += (len(m) - 1) * tiles * H_kv
        rows += sum(news[b] for b in m) if tiles else 0
    return rows if less >= least else 0


def joined(sdv, c, table, lens, news, group, M, H, D, ws, seen=None):
    """Runs a call and returns the number of query rows that its plan gave a prefix (-7: it did not look)."""
    ws.view(torch.int32)[1] = -7
    q = torch.zeros(len(lens), M, H, D, device="cuda") if seen is None else seen
    out = torch.full_like(q, 123.0)
    sdv.paged_attn_shared(q, c, table, i32(lens), i32(group), out, ws, n_new=i32(news))
    status_ok()
    return int(ws.view(torch.int32)[1]), out


@pytest.mark.parametrize("seed", range(12))
def test_what_is_shared(sdv, seed):
    """Groups of every kind over random tables: the plan gives a prefix to the rows that the tables say, and to no others."""
    rng = np.random.default_rng(300 + seed)
    P, H_kv, D = [(16, 2, 64), (8, 1, 128), (64, 2, 64), (128, 1, 64), (32, 3, 128), (16, 1, 256)][seed % 6]
    B, M, n_pages, width = int(rng.integers(2, 40)), 3, 300, 1024 // P
    k, v = (torch.randn(n_pages, H_kv, P, D, device="cuda").half() for _ in range(2))
    pages = sdv.KvPages(k, v)
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(B, M, 2 * H_kv, H_kv, D))
    some = 0
    for _ in range(10):
        lens = rng.integers(0, width * P - M + 1, B)
        news = rng.integers(0, M + 1, B)
        group = rng.integers(-1, max(1, B // 3), B)
        table = rng.integers(0, n_pages, (B, width)).astype(np.int32)
        for g in range(B):  # members share a random number of slots with the first one
            m = np.flatnonzero(group == g)
            for b in m[1:]:
                n = int(rng.integers(0, width + 1))
                table[b, :n] = table[m[0], :n]
        want = expected(table, lens, news, group, P, H_kv, n_pages, 1)
        some += want > 0
        got, out = joined(sdv, pages, torch.tensor(table).cuda(), lens, news, group, M, 2 * H_kv, D, ws, torch.randn(B, M, 2 * H_kv, D, device="cuda"))
        assert got == want
        for b in range(B):  # (the sums over random rows are other tests')
            assert torch.all(out[b, int(news[b]):] == 123.0) and torch.all(torch.isfinite(out[b]))
    assert some >= 3


@pytest.mark.parametrize("news,group,rows", [([2, 2, 2], [0, 0, 0], 6), ([2, 0, 1], [2, 2, 2], 3), ([2, 2, 2], [0, 0, -1], 4), ([0, 2, 1], [0, 0, 0], 3),
                                             ([2, 2, 2], [0, 1, 2], 0), ([2, 2, 2], [-1, -1, -1], 0), ([1, 0, 0], [0, 0, 0], 0)])
def test_who_joins_a_prefix(sdv, news, group, rows):
    k = torch.randn(20, 1, 16, 64, device="cuda").half()
    table = torch.tensor([[0, 1, 2, 3, 4, 5 + b] for b in range(3)], dtype=torch.int32).cuda()
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(3, 2, 1, 1, 64))
    assert joined(sdv, sdv.KvPages(k, k), table, [80, 85, 81], news, group, 2, 1, 64, ws)[0] == rows


@pytest.mark.parametrize("tiles", [29, 30, 31, 1 << 20])
def test_the_least_that_a_prefix_has_to_save(sdv, tiles):
    """3 other members of 2 heads by 5 tiles are 30: up to that least number they share; nobody looks where the tables (6 tiles)
    cannot hold as much."""
    k = torch.randn(60, 2, 8, 64, device="cuda").half()
    table = torch.arange(49, dtype=torch.int32).repeat(4, 1).cuda()
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(4, 2, 4, 2, 64))
    lens = [320, 321, 383, 320]
    try:
        sdv.debug_share_from(tiles)
        got = joined(sdv, sdv.KvPages(k, k), table, lens, [2, 1, 2, 2], [1] * 4, 2, 4, 64, ws)[0]
    finally:
        sdv.debug_share_from(1)
    assert got == (7 if tiles <= 30 else 0 if tiles <= 36 else -7)


@pytest.mark.parametrize("rows,held,got", [(8000, 16000, 4), (7999, 16000, 0), (8000, 15936, -7), (15000, 15936, -7), (15000, 16000, 4)])
def test_the_numbers_from_which_a_batch_shares(sdv, rows, held, got):
    """Three other members of 8 heads: 125 tiles of 64 rows are 3000, and tables of 250 tiles could hold 6000."""
    k = torch.randn(1, 8, 64, 64, device="cuda").half()
    table = torch.zeros(4, held // 64, dtype=torch.int32, device="cuda")
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(4, 1, 8, 8, 64))
    try:
        sdv.debug_share_from(0)
        assert joined(sdv, sdv.KvPages(k, k), table, [rows] * 4, [1] * 4, [0] * 4, 1, 8, 64, ws)[0] == got
    finally:
        sdv.debug_share_from(1)


def test_no_ticket_is_left(sdv):
    """Every CTA of the own rows' launch takes the ticket that the plan releases for it, whatever its grid is (two CTAs per SM or one), with and
    without programmatic launches; the same bits either way."""
    ws = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(5, 2, 16, 2, 256))
    try:
        for D, H in ((64, 4), (256, 4), (128, 16), (64, 16), (128, 2)):
            rng = np.random.default_rng(D + H)
            lens, news = [320, 700, 333, 390, 41], [2, 1, 2, 2, 2]
            c = Cache(sdv, rng, lens, news, 2, 2, D, 16, "f16")
            share(c, {(0, 1, 2, 3): 20})
            q = rng.standard_normal((5, 2, H, D)).astype(np.float32)
            outs = []
            for on in (1, 0, 1):
                sdv.set_pdl(on)
                out = torch.full(q.shape, 123.0, device="cuda")
                sdv.paged_attn_shared(cuda(q), c.pages, c.table, i32(lens), i32([0, 0, 0, 0, -1]), out, ws, n_new=i32(news))
                status_ok()
                head = ws.view(torch.int32)[:64 + 2 * torch.cuda.get_device_properties(0).multi_processor_count]
                assert int(head[0]) == 0 and int(head[1]) == 7 and torch.all(head[64:] == 0)
                outs.append(out)
            assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
            compare(outs[0], c, q, lens, news)
    finally:
        sdv.set_pdl(1)
