"""Rotary positions of rows and of a batch's new rows on their way into pages, against plain forms in 64 bits or more:
layouts, parts of heads, stretched frequencies, positions up to 2^31, trees, strides, in place, what is left alone."""
import numpy as np
import pytest
import torch

import _paged_plain as paged
import _samples_plain as plain
from _util import cuda, host, status_ok
from test_gpu_paged import TYPES, Cache, binary, i32

pytestmark = pytest.mark.gpu

EDEVICE = 5
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gb300 as m
    m.lib()
    return m


KINDS = [dict(), dict(interleaved=True), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0, interleaved=True),
         dict(scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0), dict(scaling="yarn", factor=32.0, original=4096, low=1.0, high=32.0)]


def ropes(sdv, rot, **kw):
    r = sdv.Rope(rot, **kw)
    f, s = plain.frequencies(rot, **{k: v for k, v in kw.items() if k != "interleaved"})
    return r, np.array(r.inv_freq), r.scale, f, s


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("N,heads,D,rot", [(1, 1, 8, 8), (3, 5, 64, 64), (7, 48, 128, 128), (700, 3, 128, 64), (5, 2, 256, 40), (2, 9, 72, 24),
                                           (65, 1, 1024, 1024), (400, 40, 64, 32)])
def test_rows(sdv, kind, N, heads, D, rot):
    rng = np.random.default_rng(N + rot)
    r, f, s, f_ref, s_ref = ropes(sdv, rot, **KINDS[kind])
    assert np.allclose(f, f_ref, rtol=1e-14, atol=0) and abs(s - s_ref) <= plain.U * s_ref
    x = rng.standard_normal((N, heads, D)).astype(np.float32)
    pos = rng.integers(0, 100000, N).astype(np.int32)
    pos[0] = 0
    out = torch.full((N, heads, D), 7.0, device="cuda")
    sdv.rope_rows(cuda(x), i32(pos), r, out)
    status_ok()
    ref, tol = plain.turn(x, pos, f, s, r.interleaved)
    assert np.all(np.abs(host(out) - ref) <= tol)
    assert np.array_equal(host(out)[..., rot:], x[..., rot:])


def test_positions_of_every_size(sdv):
    """Powers of two and their neighbours up to 2^31 - 1, negative ones, in both layouts."""
    pos = np.array(sorted({max(-2 ** 31, min(2 ** 31 - 1, s * (2 ** k + d))) for k in range(32) for d in (-1, 0, 1) for s in (-1, 1)}), np.int64)
    x = np.random.default_rng(1).standard_normal((len(pos), 2, 128)).astype(np.float32)
    for inter in (False, True):
        r = sdv.Rope(128, base=500000.0, interleaved=inter)
        out = torch.empty(x.shape, device="cuda")
        sdv.rope_rows(cuda(x), i32(pos), r, out)
        ref, tol = plain.turn(x, pos, np.array(r.inv_freq), 1.0, inter)
        # (the reference's own angle: 2^31 radians in 64 or 113 bits of mantissa)
        assert np.all(np.abs(host(out) - ref) <= tol + 2.0 ** -31 * np.abs(x).sum(-1, keepdims=True))
    status_ok()


def test_given_frequencies(sdv):
    f = [0.1 * (i + 1) for i in range(8)]
    r = sdv.Rope(16, inv_freq=f, scale=2.5)
    x = np.random.default_rng(2).standard_normal((9, 3, 32)).astype(np.float32)
    pos = np.arange(9, dtype=np.int32) * 1000
    out = torch.empty(x.shape, device="cuda")
    sdv.rope_rows(cuda(x), i32(pos), r, out)
    ref, tol = plain.turn(x, pos, np.array(f), 2.5, False)
    assert np.all(np.abs(host(out) - ref) <= tol)
    status_ok()


@pytest.mark.parametrize("inter", [False, True])
def test_rows_in_place_and_of_strides(sdv, inter):
    """Columns of a fused projection, turned where they are; the columns beside them are left alone."""
    rng = np.random.default_rng(3)
    line = rng.standard_normal((33, 12, 64)).astype(np.float32)
    t = cuda(line)
    r = sdv.Rope(32, interleaved=inter)
    pos = rng.integers(0, 5000, 33).astype(np.int32)
    sdv.rope_rows(t[:, 4:9], i32(pos), r, t[:, 4:9])
    got = host(t)
    ref, tol = plain.turn(line[:, 4:9], pos, np.array(r.inv_freq), 1.0, inter)
    assert np.all(np.abs(got[:, 4:9] - ref) <= tol)
    assert np.array_equal(got[:, :4], line[:, :4]) and np.array_equal(got[:, 9:], line[:, 9:])
    status_ok()


def test_rows_of_nan_and_infinity_stay_in_their_pairs(sdv):
    x = np.ones((2, 2, 64), np.float32)
    x[0, 0, 3], x[1, 1, 40] = np.nan, np.inf
    out = torch.empty(x.shape, device="cuda")
    sdv.rope_rows(cuda(x), i32([5, 6]), sdv.Rope(64), out)
    bad = ~np.isfinite(host(out))
    want = np.zeros(x.shape, bool)
    want[0, 0, [3, 35]] = want[1, 1, [8, 40]] = True
    assert np.array_equal(bad, want)
    status_ok()


def check_append(sdv, seed, lens, news, M, H, H_kv, D, P, dtype, rot, nhd=False, parents=None, in_place=False, fused=True, **kw):
    rng = np.random.default_rng(seed)
    B = len(lens)
    c = Cache(sdv, rng, lens, news, M, H_kv, D, P, dtype, nhd)
    r = sdv.Rope(rot, **kw)
    before = [x.clone() if x is not None else None for x in (c.k, c.v, c.ks, c.vs)]
    line = rng.standard_normal((B, M, H + 2 * H_kv, D)).astype(np.float32)
    t = cuda(line)
    q, k, v = t[:, :, :H], t[:, :, H:H + H_kv], t[:, :, H + H_kv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    out = (q if in_place else torch.full((B, M, H, D), 55.0, device="cuda")) if H else None
    sdv.paged_append_rope(q if H else None, k, v, c.pages, c.table, i32(lens), r, out, n_new=i32(news) if news is not None else None,
                          parent=i32(parents) if parents is not None else None)
    status_ok()
    freq = np.array(r.inv_freq)
    table = host(c.table)
    touched = np.zeros((c.k.shape[0], P), bool)
    got_q = host(out) if H else None
    for b, L in enumerate(lens):
        n = news[b]
        depth = [len(paged.path_of(parents[b], i)) - 1 for i in range(n)] if parents is not None else list(range(n))
        pos = L + np.array(depth, np.int64)
        if H:
            ref, tol = plain.turn(line[b, :n, :H], pos, freq, r.scale, r.interleaved)
            assert np.all(np.abs(got_q[b, :n] - ref) <= tol)
            assert np.array_equal(got_q[b, n:], line[b, n:, :H]) if in_place else np.all(got_q[b, n:] == 55.0)
        for i in range(n):
            touched[table[b, (L + i) // P], (L + i) % P] = True
        if n == 0:
            continue
        rk, tk = plain.turn(line[b, :n, H:H + H_kv], pos, freq, r.scale, r.interleaved)
        rv, tv = line[b, :n, H + H_kv:].astype(np.float64), np.zeros((n, H_kv, D))
        gk, gv = (x.transpose(1, 0, 2) for x in c.rows(b, L, L + n))
        for got, ref, tol, s in ((gk, rk, tk, c.ks), (gv, rv, tv, c.vs)):
            if dtype == "i8":
                scale = np.abs(ref).max(-1, keepdims=True) / 127
                off = tol.max(-1, keepdims=True) / 127 + 2 * plain.U * scale  # of the scale
                assert np.all(np.abs(got - ref) <= (scale + off) / 2 + tol + 128 * off + 4 * plain.U * np.abs(ref))
            else:
                assert np.all(np.abs(got - ref) <= tol + HALF[dtype] * (np.abs(ref) + tol) + TINY[dtype])
    # every other row of the pool is as it was
    for x, y in zip((c.k, c.v, c.ks, c.vs), before):
        if x is not None:
            x, y = host(x.float()), host(y.float())
            same = (x == y) | (np.isnan(x) & np.isnan(y))
            assert np.all(same.reshape(same.shape[:3] + (-1,)).all(-1).transpose(0, 2, 1)[~touched])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("H,H_kv,D,P,M,rot,nhd", [(8, 2, 128, 16, 1, 128, False), (40, 8, 128, 64, 5, 64, True), (3, 3, 64, 8, 3, 24, True),
                                                  (4, 1, 256, 32, 2, 256, False), (0, 5, 64, 16, 7, 64, False), (7, 1, 128, 192, 70, 8, False)])
def test_append(sdv, dtype, H, H_kv, D, P, M, rot, nhd):
    lens = [0, 1, P - 1, P, 63, 64, 1000]
    news = [M, max(1, M - 1), M, 0, 1, M, M // 2]
    for inter in (False, True):
        check_append(sdv, M + rot, lens, news, M, H, H_kv, D, P, dtype, rot, nhd, interleaved=inter, in_place=inter, fused=not inter or H > 0)


@pytest.mark.parametrize("dtype", ["f16", "i8"])
@pytest.mark.parametrize("M", [2, 11, 16])
def test_append_of_trees(sdv, dtype, M):
    parents = [binary(M), [-1] + [0] * (M - 1), list(range(-1, M - 1)), [-1] + [max(0, i - 2) for i in range(1, M)]]
    check_append(sdv, M, [0, 77, 640, 5], [M, M, M - 1, M], M, 8, 4, 128, 16, dtype, 128, parents=parents, scaling="yarn", factor=8.0, original=4096,
                 low=1.0, high=32.0)


def test_append_of_16_bit_rows_without_a_turn_is_paged_append(sdv):
    """At position 0 nothing turns: the same bits as sd_paged_append, 8-bit rows too."""
    for dtype in TYPES:
        rng = np.random.default_rng(4)
        a = Cache(sdv, rng, [0] * 3, [1] * 3, 1, 2, 128, 16, dtype)
        b = Cache(sdv, np.random.default_rng(4), [0] * 3, [1] * 3, 1, 2, 128, 16, dtype)
        k, v = (cuda(rng.standard_normal((3, 1, 2, 128)).astype(np.float32)) for _ in range(2))
        sdv.paged_append(k, v, a.pages, a.table, i32([0] * 3))
        sdv.paged_append_rope(None, k, v, b.pages, b.table, i32([0] * 3), sdv.Rope(128), None)
        for x, y in ((a.k, b.k), (a.v, b.v), (a.ks, b.ks), (a.vs, b.vs)):
            if x is not None:
                assert torch.equal(torch.nan_to_num(x.float(), 9.0), torch.nan_to_num(y.float(), 9.0))
    status_ok()


def test_append_of_infinite_rows(sdv):
    """8-bit rows: an infinity or NaN is the row's scale, as in sd_paged_append."""
    c = Cache(sdv, np.random.default_rng(5), [10, 10], [2, 2], 2, 1, 64, 16, "i8")
    k = torch.ones(2, 2, 1, 64, device="cuda")
    k[0, 0, 0, 60], k[1, 1, 0, 60] = float("inf"), float("nan")  # (behind the turned part)
    sdv.paged_append_rope(None, k, k.clone(), c.pages, c.table, i32([10, 10]), sdv.Rope(32), None)
    status_ok()
    t = host(c.table)
    for s in (c.ks, c.vs):
        s = host(s)
        assert np.isinf(s[t[0, 0], 0, 10]) and np.isfinite(s[t[0, 0], 0, 11])
        assert np.isfinite(s[t[1, 0], 0, 10]) and np.isnan(s[t[1, 0], 0, 11])


def test_bad_lengths_pages_and_trees_are_skipped_and_recorded(sdv):
    def run(lens=(5, 5), news=(2, 2), spoil=None, parent=None):
        c = Cache(sdv, np.random.default_rng(6), [5, 5], [2, 2], 2, 2, 64, 16, "f16")
        if spoil is not None:
            c.table[0, 0] = spoil
        before = c.k.clone()
        q = torch.ones(2, 2, 4, 64, device="cuda")
        out = torch.full((2, 2, 4, 64), 9.0, device="cuda")
        kv = torch.ones(2, 2, 2, 64, device="cuda")
        sdv.paged_append_rope(q, kv, kv, c.pages, c.table, i32(lens), sdv.Rope(64), out, n_new=i32(news), parent=parent)
        same = torch.equal(torch.nan_to_num(before, 3.0)[c.table[0, 0].clamp(min=0) % before.shape[0]],
                           torch.nan_to_num(c.k, 3.0)[c.table[0, 0].clamp(min=0) % before.shape[0]])
        return sdv.device_status(), out, same

    assert run()[0] == 0
    for bad in (dict(lens=(-1, 5)), dict(lens=(1000, 5)), dict(news=(3, 2)), dict(news=(-1, 2))):
        st, out, same = run(**bad)
        assert st == EDEVICE and same and torch.all(out[0] == 9.0) and torch.all(out[1] != 9.0), bad
    for page in (-1, 10 ** 6):
        st, out, _ = run(spoil=page)
        assert st == EDEVICE and torch.all(out != 9.0)  # its queries are turned all the same
    st, out, _ = run(parent=i32([[-1, 1], [-1, 0]]))
    assert st == EDEVICE and torch.all(torch.isfinite(out))


def test_append_on_another_stream_and_replayed(sdv):
    """On a stream of its own, captured and replayed with other lengths and rows."""
    lens, M = [3, 40], 2
    c = Cache(sdv, np.random.default_rng(7), [3 + 8, 40 + 8], [M, M], M, 2, 128, 16, "bf16")
    r = sdv.Rope(128)
    line = torch.randn(2, M, 8, 128, device="cuda")
    q_out, L = torch.zeros(2, M, 4, 128, device="cuda"), i32(lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sdv.paged_append_rope(line[:, :, :4], line[:, :, 4:6], line[:, :, 6:], c.pages, c.table, L, r, q_out)
        for add in (0, 5, 8):
            L.copy_(i32([x + add for x in lens]))
            line.copy_(torch.randn(line.shape, device="cuda"))
            g.replay()
            s.synchronize()
            for b in range(2):
                pos = lens[b] + add + np.arange(M)
                ref, tol = plain.turn(host(line)[b, :, :4], pos, np.array(r.inv_freq), 1.0, False)
                assert np.all(np.abs(host(q_out)[b] - ref) <= tol)
                rk, tk = plain.turn(host(line)[b, :, 4:6], pos, np.array(r.inv_freq), 1.0, False)
                k, v = (x.transpose(1, 0, 2) for x in c.rows(b, int(pos[0]), int(pos[0]) + M))
                assert np.all(np.abs(k - rk) <= tk + HALF["bf16"] * (np.abs(rk) + tk))
                assert np.all(np.abs(v - host(line)[b, :, 6:]) <= HALF["bf16"] * np.abs(v) + 1e-30)
    status_ok()
