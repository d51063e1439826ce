"""Tokens drawn from rows of logits against the order and sums in 64 bits: every filter alone and together, ties, masks,
infinities, vocabularies from one token on, settings per row, strides, and rows that have no answer."""

import numpy as np
import pytest
import torch

import _samples_plain as plain
from _util import cuda, host, status_ok

pytestmark = pytest.mark.gpu

EDEVICE = 5


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gb300 as m
    m.lib()
    return m


def run(sdv, l, u, T=None, k=None, p=None, low=None, probs=True):
    N, V = l.shape
    l = l if isinstance(l, torch.Tensor) else cuda(l.astype(np.float32))
    tokens, prob = torch.full((N,), -7, dtype=torch.int32, device="cuda"), torch.full((N,), 7.0, device="cuda")
    all_ = torch.full((N, V), 7.0, device="cuda") if probs else None
    f = lambda v: None if v is None else cuda(np.asarray(v, np.float32))  # noqa: E731
    sdv.sample(l, f(u), tokens, temperature=f(T), top_k=None if k is None else cuda(np.asarray(k, np.int32)), top_p=f(p), min_p=f(low), prob=prob,
               probs=all_)
    return host(tokens), host(prob), host(all_) if probs else None


def check(sdv, l, u, T=None, k=None, p=None, low=None, probs=True):
    N = l.shape[0]
    tokens, prob, all_ = run(sdv, l, u, T, k, p, low, probs)
    status_ok()
    at = lambda v, n, off: off if v is None else v[n]  # noqa: E731
    h = host(l) if isinstance(l, torch.Tensor) else l.astype(np.float32)
    for n in range(N):
        plain.check_row(h[n], float(np.float32(u[n])), float(np.float32(at(T, n, 1.0))), int(at(k, n, 0)), float(np.float32(at(p, n, 1.0))),
                        float(np.float32(at(low, n, 0.0))), int(tokens[n]), float(prob[n]), all_[n].astype(np.float64) if probs else None)
    return tokens


def logits(rng, N, V, kind):
    x = rng.standard_normal((N, V)) * 2.0
    if kind == "coarse":  # many equal ones
        x = np.round(x * 2) / 2
    elif kind == "equal":
        x = np.full((N, V), 1.5)
    elif kind == "two":  # tiny differences beside a large logit: equal distances, different logits
        x = rng.standard_normal((N, V)) * 1e-9
        x[:, rng.integers(V)] = 1e4
    elif kind == "peaked":
        x[:, rng.integers(V)] += 30.0
    elif kind == "masked":
        x[rng.random((N, V)) < 0.7] = -np.inf
        x[:, rng.integers(V)] = 0.5
    elif kind == "lowest":
        x[rng.random((N, V)) < 0.7] = np.finfo(np.float32).min
        x[:, rng.integers(V)] = 0.5
    elif kind == "far":
        x = x * 1e6
    elif kind == "near":
        x = 5.0 + x * 1e-6
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["plain", "coarse", "equal", "two", "peaked", "masked", "lowest", "far", "near"])
@pytest.mark.parametrize("V", [1, 2, 17, 255, 1000, 2049, 8193, 40001])
def test_filters(sdv, V, kind):
    rng = np.random.default_rng(V)
    settings = [(1.0, 0, 1.0, 0.0), (0.7, 1, 1.0, 0.0), (1.0, 40, 1.0, 0.0), (1.0, max(1, V // 2), 1.0, 0.0), (1.0, V, 1.0, 0.0), (1.0, V + 5, 0.9, 0.0),
                (0.9, 0, 0.9, 0.0), (1.5, 0, 0.3, 0.0), (1.0, 0, 0.999, 0.0), (1.0, 0, 1e-9, 0.0), (1.0, 0, 1.0, 0.05), (1.0, 0, 1.0, 1.0),
                (0.8, 300, 0.95, 0.0), (0.8, 300, 0.95, 0.02), (0.0, 0, 1.0, 0.0), (0.0, 50, 0.5, 0.5), (10.0, 0, 0.9, 0.5), (0.05, 7, 0.99, 0.0)]
    T, k, p, low = (list(x) for x in zip(*settings))
    l = logits(rng, len(settings), V, kind)
    for probs in (True, False):
        u = np.minimum(rng.random(len(settings)).astype(np.float32), np.float32(1 - 2.0 ** -24))
        u[0], u[1] = 0.0, 1 - 2.0 ** -24
        check(sdv, l, u, T, k, p, low, probs)


@pytest.mark.parametrize("V", [151936, 151937, 360448])
def test_whole_vocabularies(sdv, V):
    rng = np.random.default_rng(5)
    for kind, T, k, p, low in (("plain", 0.8, 50, 0.95, 0.0), ("plain", 1.0, 0, 0.9, 0.0), ("coarse", 1.0, 1000, 0.99, 0.01), ("equal", 1.0, 0, 0.5, 0.0),
                               ("masked", 1.2, 0, 1.0, 0.1), ("two", 1.0, V - 3, 1.0, 0.0)):
        N = 5
        check(sdv, logits(rng, N, V, kind), rng.random(N).astype(np.float32) * 0.999, [T] * N, [k] * N, [p] * N, [low] * N)


@pytest.mark.parametrize("N,V", [(320, 151936), (320, 151937), (160, 100001), (70, 151937), (70, 360448)])
def test_many_rows_of_whole_vocabularies(sdv, N, V):
    """Rows that share the GPU with so many others that one, two or four CTAs read them again and again: the same tokens and
    probabilities as alone, and right."""
    rng = np.random.default_rng(N)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    l = torch.randn(N, V, generator=gen, device="cuda") * 2
    l[1::4] = torch.round(l[1::4] * 4) / 4
    l[2::8] = -float("inf")
    l[2::8, 77:1000] = 0.25
    l[3, 5] = l[3, 9] = float("inf")
    l[5] = float("nan")
    l[5, 11] = -1.0
    u = rng.random(N).astype(np.float32) * 0.999
    T = (0.5 + rng.random(N)).astype(np.float32)
    k = rng.choice([0, 0, 1, 30, 300, 5000], N).astype(np.int32)
    p = rng.choice([1.0, 0.9, 0.3], N).astype(np.float32)
    low = rng.choice([0.0, 0.0, 0.02], N).astype(np.float32)
    for with_p in (True, False):
        args = (T, k, p if with_p else None, low)
        tokens, prob, _ = run(sdv, l, u, *args, probs=False)
        status_ok()
        for n in list(range(12)) + [N - 1]:
            alone, prob1, q = run(sdv, l[n:n + 1], u[n:n + 1], *(x[n:n + 1] if x is not None else None for x in args))
            assert alone[0] == tokens[n] and prob1[0] == prob[n]
            plain.check_row(host(l[n]), float(u[n]), float(T[n]), int(k[n]), float(p[n]) if with_p else 1.0, float(low[n]), int(tokens[n]),
                            float(prob[n]), q[0].astype(np.float64))
    status_ok()


@pytest.mark.parametrize("V,N", [(1000, 64), (30000, 64), (30000, 2000)])
def test_nuclei_that_end_at_a_border(sdv, V, N):
    """Levels of equal logits, and top-p within some roundings of the sum down to a level's end: the histogram's sums alone do not
    tell on which side of it the nucleus ends."""
    rng = np.random.default_rng(V)
    l, p = np.zeros((N, V), np.float32), np.zeros(N, np.float32)
    for n in range(N):
        cut = np.sort(rng.choice(np.arange(1, V), 4, replace=False))
        level = -np.cumsum(rng.choice([0.01, 0.3, 1.0, 2.5], 5)).astype(np.float32)
        l[n] = rng.permutation(level[np.searchsorted(cut, np.arange(V), side="right")])
        w = np.exp(np.sort(l[n].astype(np.float64))[::-1] - l[n].max())
        share = np.cumsum(w)[cut[rng.integers(4)] - 1] / w.sum()
        p[n] = np.float32(share) + np.float32(rng.integers(-3, 4)) * np.spacing(np.float32(share))
    check(sdv, l, rng.random(N).astype(np.float32) * 0.999, p=np.minimum(p, 1))
    if N < 100:
        check(sdv, l, rng.random(N).astype(np.float32) * 0.999, p=np.minimum(p, 1), k=[V - 1] * N, probs=False)


@pytest.mark.parametrize("N", [6, 160])
def test_low_temperatures(sdv, N):
    """A token and, 9.5 to 13 temperatures behind it, all others: at such a temperature that distance is within one of the first
    histogram's bins, where the others' parts are rounded away, although together they weigh as much or more."""
    rng = np.random.default_rng(N)
    V, T = 151936, np.float32([1e-3, 3e-4, 1e-6, 5e-3, 1e-2, 1e-3])[np.arange(N) % 6]
    far = np.float32([9.5, 10.6, 11.3, 12.0, 10.6, 13.0])[np.arange(N) % 6]
    l = -T[:, None] * (far[:, None] + 0.2 * rng.random((N, V)))
    top = rng.integers(V, size=N)
    l[np.arange(N), top] = 0.0
    l = l.astype(np.float32)
    u = rng.random(N).astype(np.float32) * 0.999
    for p in (0.3, 0.5, 0.8, 0.999):
        for k, low in ((0, 0.0), (100000, 0.0), (0, 1e-5)):
            tokens, prob, _ = run(sdv, l, u, T, [k] * N, [p] * N, [low] * N, probs=False)
            status_ok()
            for n in range(6):
                tok1, prob1, q = run(sdv, l[n:n + 1], u[n:n + 1], T[n:n + 1], [k], [p], [low])
                assert tok1[0] == tokens[n] and prob1[0] == prob[n]
                plain.check_row(l[n], float(u[n]), float(T[n]), k, float(np.float32(p)), float(np.float32(low)), int(tokens[n]), float(prob[n]),
                                q[0].astype(np.float64))
    status_ok()


def test_ties_go_to_the_lower_index(sdv):
    l = np.array([[1, 3, 3, 2, 3, 3, 0, 3.0]] * 8, np.float32)
    u = np.arange(8) / 8 + 1 / 16
    _, _, q = run(sdv, l, u, k=[1, 2, 3, 4, 5, 6, 7, 8])
    for n in range(8):
        assert list(np.nonzero(q[n])[0]) == sorted([1, 2, 4, 5, 7, 3, 0, 6][:n + 1])
    # half of two equal tokens is the first of them, exactly; a little more is both
    _, _, q = run(sdv, np.array([[5, 5.0]] * 3, np.float32), [0.9] * 3, p=[0.5, np.nextafter(np.float32(0.5), np.float32(1)), 1.0])
    assert [list(np.nonzero(x)[0]) for x in q] == [[0], [0, 1], [0, 1]]
    tokens, _, q = run(sdv, np.array([[-0.0, 0.0, -0.0]], np.float32), [0.0], k=[2])
    assert list(np.nonzero(q[0])[0]) == [0, 1] and tokens[0] == 0
    # the first token whose running sum is above u: at 1/2 of two equal ones the second
    tokens, prob, _ = run(sdv, np.array([[5, 5.0]] * 2, np.float32), [0.5, np.nextafter(np.float32(0.5), np.float32(0))])
    assert list(tokens) == [1, 0] and np.all(prob == 0.5)
    status_ok()


def test_greedy(sdv):
    rng = np.random.default_rng(6)
    l = logits(rng, 16, 5000, "coarse")
    tokens, prob, _ = run(sdv, l, rng.random(16), T=[0.0] * 16)
    assert np.array_equal(tokens, l.argmax(1)) and np.all(prob == 1.0)
    status_ok()


def test_infinities_and_nan(sdv):
    inf = np.inf
    l = np.array([[0, -inf, np.nan, 1], [inf, 0, inf, np.nan], [-inf, -inf, 3, -inf], [np.nan, 2, np.nan, 2], [3.4e38, -3.4e38, 3.4e38, 0]], np.float32)
    tokens, prob, q = run(sdv, l, [0.99, 0.75, 0.0, 0.4, 0.6])
    status_ok()
    assert list(tokens) == [3, 2, 2, 1, 2]
    assert np.array_equal(q > 0, [[1, 0, 0, 1], [1, 0, 1, 0], [0, 0, 1, 0], [0, 1, 0, 1], [1, 0, 1, 0]])
    for low in (0.5, 1.0):
        _, _, q = run(sdv, l, [0.5] * 5, low=[low] * 5, k=[3] * 5, p=[0.99] * 5)
        assert np.all(q[1, [0, 2]] == 0.5) and np.all(q[4, [0, 2]] == 0.5)
    status_ok()


def test_rows_without_an_answer(sdv):
    """A setting out of range, or no token at all: -1, 0 and zeros, recorded; the rows beside them are right."""
    l = np.tile(np.arange(100, dtype=np.float32) / 10, (12, 1))
    l[0] = -np.inf
    l[1] = np.nan
    ok = dict(u=[0.5] * 12, T=[1.0] * 12, k=[0] * 12, p=[1.0] * 12, low=[0.0] * 12)
    for name, n, v in (("T", 2, -1.0), ("T", 3, np.nan), ("T", 4, np.inf), ("k", 5, -1), ("p", 6, 0.0), ("p", 7, 1.5), ("low", 8, -0.1), ("low", 9, 1.1),
                       ("u", 10, 1.0)):
        ok[name][n] = v
    tokens, prob, q = run(sdv, l, **ok)
    assert sdv.device_status() == EDEVICE and sdv.device_status() == 0
    assert np.all(tokens[:11] == -1) and np.all(prob[:11] == 0) and np.all(q[:11] == 0)
    plain.check_row(l[11], 0.5, 1.0, 0, 1.0, 0.0, int(tokens[11]), float(prob[11]), q[11].astype(np.float64))
    for bad in (np.nan, -0.5, 2.0):
        tokens, _, _ = run(sdv, l[11:], [bad])
        assert tokens[0] == -1 and sdv.device_status() == EDEVICE
    # temperatures at the ends of the range: the smallest keep the equal largest, the largest make all tokens equal
    l = np.array([[1, 2, 2, 0]] * 2, np.float32)
    tokens, _, q = run(sdv, l, [0.5, 0.1], T=[1e-45, 3e38])
    status_ok()
    assert np.allclose(q, [[0, 0.5, 0.5, 0], [0.25] * 4]) and list(tokens) == [2, 0]


def test_a_row_does_not_depend_on_its_batch(sdv):
    rng = np.random.default_rng(7)
    l, u = logits(rng, 40, 30000, "plain"), rng.random(40)
    T, k, p = list(0.5 + rng.random(40)), [0, 100] * 20, [0.9, 1.0, 0.95, 0.5] * 10
    a = run(sdv, l, u, T, k, p)
    for n in (0, 1, 7, 39):
        b = run(sdv, l[n:n + 1], u[n:n + 1], T[n:n + 1], k[n:n + 1], p[n:n + 1])
        for x, y in zip(a, b):
            assert np.array_equal(x[n:n + 1], y)
    for x, y in zip(a, run(sdv, l, u, T, k, p)):
        assert np.array_equal(x, y)
    status_ok()


@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_rows_of_any_stride(sdv, off):
    """Rows that begin at any element, and probabilities written into columns of a wider tensor."""
    rng = np.random.default_rng(8)
    N, V = 6, 4099
    wide = torch.full((N, V + 9), float("inf"), device="cuda")
    wide[:, off:off + V] = cuda(logits(rng, N, V, "plain"))
    l = wide[:, off:off + V]
    to = torch.full((N, V + 7), 3.0, device="cuda")
    tokens, prob = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros(N, device="cuda")
    u = rng.random(N).astype(np.float32)
    sdv.sample(l, cuda(u), tokens, top_p=torch.full((N,), 0.9, device="cuda"), prob=prob, probs=to[:, off:off + V])
    status_ok()
    t, q, pr = host(tokens), host(to), host(prob)
    for n in range(N):
        plain.check_row(host(l)[n], float(u[n]), 1.0, 0, float(np.float32(0.9)), 0.0, int(t[n]), float(pr[n]), q[n, off:off + V].astype(np.float64))
    assert np.all(q[:, :off] == 3.0) and np.all(q[:, off + V:] == 3.0)


def test_frequencies_of_draws(sdv):
    """300000 draws of 16 tokens: every count within 5 sigma of its probability, and forbidden tokens never."""
    rng = np.random.default_rng(9)
    l = logits(rng, 1, 16, "plain")
    l[0, 3] = -np.inf
    n = 300000
    tokens, _, _ = run(sdv, torch.tensor(l).cuda().expand(n, 16).contiguous(), rng.random(n), k=[12] * n, probs=False)
    status_ok()
    w = np.exp(l[0].astype(np.float64) - l.max())
    w[np.argsort(-w)[12:]] = 0
    p = w / w.sum()
    got = np.bincount(tokens, minlength=16)
    assert np.all(np.abs(got - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1e-9)


def test_captured_and_on_another_stream(sdv):
    rng = np.random.default_rng(10)
    l, u = torch.empty(4, 9000, device="cuda"), torch.empty(4, device="cuda")
    tokens, prob = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    k = torch.full((4,), 30, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        l.zero_()
        u.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sdv.sample(l, u, tokens, top_k=k, prob=prob)
        for _ in range(3):
            l.copy_(cuda(logits(rng, 4, 9000, "plain")))
            u.copy_(cuda(rng.random(4).astype(np.float32) * 0.99))
            g.replay()
            s.synchronize()
            for n in range(4):
                plain.check_row(host(l)[n], float(u[n]), 1.0, 30, 1.0, 0.0, int(tokens[n]), float(prob[n]), None)
    status_ok()


def test_two_streams_at_once(sdv):
    rng = np.random.default_rng(12)
    streams = [torch.cuda.Stream() for _ in range(2)]
    l = [cuda(logits(rng, 20, 60000, "plain")) for _ in range(2)]
    u = [cuda(rng.random(20).astype(np.float32) * 0.999) for _ in range(2)]
    p = torch.full((20,), 0.9, device="cuda")
    out = [(torch.zeros(20, dtype=torch.int32, device="cuda"), torch.zeros(20, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, x, y, o in zip(streams, l, u, out):
            with torch.cuda.stream(s):
                sdv.sample(x, y, o[0], top_p=p, prob=o[1])
    torch.cuda.synchronize()
    status_ok()
    for x, y, o in zip(l, u, out):
        for n in range(20):
            plain.check_row(host(x)[n], float(y[n]), 1.0, 0, float(np.float32(0.9)), 0.0, int(o[0][n]), float(o[1][n]), None)


def test_a_drafter_that_samples(sdv):
    """Its distributions are the q of the acceptance: with the target's logits the same, every draft is kept."""
    rng = np.random.default_rng(11)
    V, K = 3000, 4
    l = cuda(logits(rng, K + 1, V, "plain"))
    drafts, q = torch.zeros(K, dtype=torch.int32, device="cuda"), torch.zeros(K, V, device="cuda")
    out, n = torch.zeros(K + 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for seed in range(20):
        sdv.sample(l[:K], cuda(rng.random(K).astype(np.float32) * 0.999), drafts, top_k=torch.full((K,), 20, dtype=torch.int32, device="cuda"), probs=q)
        sdv.accept_sample_topk(l, K, drafts, out, n, top_k=20, q_probs=q, seed=seed)
        assert abs(float(q.sum()) - K) < 1e-4
        # p = q up to rounding: u q < p fails for u within 2^-20 of 1 alone
        assert int(n) == K + 1 and torch.equal(out[:K], drafts)
    status_ok()


@pytest.mark.parametrize("change", [dict(u=torch.float64), dict(tokens=torch.int64), dict(temperature=torch.float16), dict(top_k=torch.float32),
                                    dict(logits=torch.bfloat16)])
def test_wrong_types_are_refused(sdv, change):
    d = dict(logits=torch.zeros(2, 50, device="cuda"), u=torch.zeros(2, device="cuda"), tokens=torch.zeros(2, dtype=torch.int32, device="cuda"),
             temperature=torch.ones(2, device="cuda"), top_k=torch.ones(2, dtype=torch.int32, device="cuda"))
    d = {k: v.to(change[k]) if k in change else v for k, v in d.items()}
    with pytest.raises(ValueError):
        sdv.sample(**d)
    with pytest.raises(ValueError):
        sdv.sample(torch.zeros(50, 2, device="cuda").t(), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"))
