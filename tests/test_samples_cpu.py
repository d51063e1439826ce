"""Rotary, shared-prefix and sampling calls refuse what they do not take before anything is launched, and the host's
tables of frequencies and turns are right (no GPU needed)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import _samples_plain as plain

EINVAL, EUNSUPPORTED = 1, 2
A = 1 << 20  # an aligned address that nothing dereferences on the host


@pytest.fixture(scope="module")
def sdv():
    from speculative_decoding_verify_gb300 import build as b
    b.build()
    import speculative_decoding_verify_gb300 as m
    m.lib()
    return m


def pages(sdv, **kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, type=0, n_pages=10, page_rows=16, H_kv=4, D=128, page_stride=4 * 16 * 128,
             head_stride=16 * 128, row_stride=128)
    d.update(kw)
    return ctypes.byref(sdv.SdKvPages(*[d[f] for f, _ in sdv.SdKvPages._fields_]))


def rope(sdv, **kw):
    d = dict(turns=A, rot=64, interleaved=0, scale=1.0)
    d.update(kw)
    return ctypes.byref(sdv.SdRope(*d.values()))


def freqs(sdv, rot, *args):
    f, s = (ctypes.c_double * (rot // 2))(), ctypes.c_float()
    code = sdv.lib().sd_rope_freqs(rot, *args, f, ctypes.byref(s))
    return code, np.array(f), float(s.value)


@pytest.mark.parametrize("rot", [2, 8, 24, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor,original,low,high", [
    ("plain", 1.0, 0, 0, 0), ("linear", 4.0, 0, 0, 0), ("ntk", 8.0, 0, 0, 0), ("bands", 8.0, 8192, 1.0, 4.0), ("yarn", 32.0, 4096, 1.0, 32.0),
    ("yarn", 1.0, 100, 0.5, 2.0), ("bands", 2.0, 1, 0.001, 0.002), ("yarn", 40.0, 5, 1.0, 32.0),
])
def test_frequencies(sdv, rot, scaling, factor, original, low, high):
    for base in (10000.0, 1000000.0, 1.5):
        code, f, s = freqs(sdv, rot, base, sdv.ROPE_SCALINGS[scaling], factor, original, low, high)
        ref, scale = plain.frequencies(rot, base, scaling, factor, original, low, high)
        assert code == 0
        assert np.all(np.abs(f - ref) <= 16 * 2.0 ** -53 * ref)
        assert s == np.float32(scale)


def test_turns_are_exact(sdv):
    """2^64 times f / 2 pi modulo 2^64, to one unit, for frequencies of every size (1 / 2 pi to 50 digits)."""
    inv = Fraction(159154943091895335768883763372514362034459645740456448747667344058896797634226535, 10 ** 81)
    f = [1.0, 0.5, 1e-3, 1e-7, 1e-20, 0.0, 3.0, 6.283185307179586, 7.5, 1000.25, 1048576.0, 2.0 ** -40, 1 / 3, -0.1, -5.5, -1e-9]
    f += list(10000.0 ** (-2.0 * np.arange(64) / 128))
    n = len(f)
    t = (ctypes.c_uint64 * n)()
    assert sdv.lib().sd_rope_turns((ctypes.c_double * n)(*f), n, t) == 0
    for x, got in zip(f, t):
        want = Fraction(x) * inv * 2 ** 64
        off = (Fraction(got) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, x


def test_frequencies_and_turns_refuse(sdv):
    L = sdv.lib()
    ok = dict(rot=64, base=1e4, scaling=4, factor=2.0, original=100.0, low=1.0, high=4.0)
    for change, code in [(dict(rot=0), EINVAL), (dict(rot=63), EINVAL), (dict(base=1.0), EINVAL), (dict(base=float("inf")), EINVAL),
                         (dict(base=float("nan")), EINVAL), (dict(scaling=5), EUNSUPPORTED), (dict(scaling=-1), EUNSUPPORTED),
                         (dict(factor=0.5), EINVAL), (dict(factor=float("nan")), EINVAL), (dict(original=0.0), EINVAL),
                         (dict(low=0.0), EINVAL), (dict(high=1.0), EINVAL), (dict(high=float("nan")), EINVAL)]:
        d = {**ok, **change}
        f, s = (ctypes.c_double * 64)(), ctypes.c_float()
        assert L.sd_rope_freqs(*d.values(), f, ctypes.byref(s)) == code, change
    f, t = (ctypes.c_double * 2)(1.0, float("nan")), (ctypes.c_uint64 * 2)(7, 7)
    assert L.sd_rope_turns(f, 2, t) == EINVAL and list(t) == [7, 7]
    assert L.sd_rope_turns((ctypes.c_double * 1)(2.0 ** 21), 1, t) == EINVAL
    assert L.sd_rope_turns(None, 2, t) == EINVAL and L.sd_rope_turns(f, 0, t) == EINVAL and L.sd_rope_turns(f, 2, None) == EINVAL


BAD_ROPES = [(dict(turns=None), EINVAL), (dict(turns=A + 8), EINVAL), (dict(rot=0), EINVAL), (dict(rot=136), EINVAL), (dict(rot=-8), EINVAL),
             (dict(rot=12), EUNSUPPORTED), (dict(rot=2), EUNSUPPORTED), (dict(interleaved=2), EINVAL), (dict(scale=float("inf")), EINVAL),
             (dict(scale=float("nan")), EINVAL)]


def rows(sdv, r, **kw):
    d = dict(x=A, xs=1024, pos=A, N=3, heads=8, D=128, out=A, os=1024)
    d.update(kw)
    return sdv.lib().sd_rope_rows(r, *d.values(), None)


def append(sdv, p, r, **kw):
    d = dict(table=A, width=4, lens=A, n_new=None, B=2, M=5, H=8, q=A, q_sb=5 * 1024, q_sm=1024, k=A, v=A, sb=5 * 512, sm=512, parent=None,
             rope=r, q_out=A, o_sb=5 * 1024, o_sm=1024)
    d.update(kw)
    return sdv.lib().sd_paged_append_rope(p, *d.values(), None)


@pytest.mark.parametrize("change,code", BAD_ROPES)
def test_bad_ropes_are_refused(sdv, change, code):
    assert rows(sdv, rope(sdv, **change)) == code
    assert append(sdv, pages(sdv), rope(sdv, **change)) == code


def test_rope_calls_refuse(sdv):
    r, p = rope(sdv), pages(sdv)
    assert rows(sdv, None) == EINVAL and append(sdv, p, None) == EINVAL and append(sdv, None, r) == EINVAL
    for change, code in [(dict(x=None), EINVAL), (dict(x=A + 4), EINVAL), (dict(pos=None), EINVAL), (dict(out=None), EINVAL), (dict(out=A + 8), EINVAL),
                         (dict(N=0), EINVAL), (dict(heads=0), EINVAL), (dict(D=0), EINVAL), (dict(D=100), EUNSUPPORTED), (dict(D=1032), EUNSUPPORTED),
                         (dict(xs=1020), EINVAL), (dict(xs=1026), EINVAL), (dict(os=1020), EINVAL), (dict(os=1025), EINVAL)]:
        assert rows(sdv, r, **change) == code, change
    for change, code in [(dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k=A + 4), EINVAL),
                         (dict(B=0), EINVAL), (dict(M=0), EINVAL), (dict(H=-1), EINVAL), (dict(width=0), EINVAL), (dict(B=1025), EUNSUPPORTED),
                         (dict(parent=A, M=17, q_sb=17 * 1024, o_sb=17 * 1024, sb=17 * 512), EUNSUPPORTED), (dict(q=None), EINVAL), (dict(q=A + 8), EINVAL),
                         (dict(q_out=None), EINVAL), (dict(q_out=A + 4), EINVAL), (dict(q_sm=1020), EINVAL), (dict(q_sm=1026), EINVAL), (dict(q_sb=1020), EINVAL),
                         (dict(o_sm=1020), EINVAL), (dict(o_sb=1022), EINVAL), (dict(sm=508), EINVAL), (dict(sb=510), EINVAL), (dict(width=1 << 28), EUNSUPPORTED)]:
        assert append(sdv, p, r, **change) == code, change
    assert append(sdv, pages(sdv, D=96), r) == EUNSUPPORTED


def shared(sdv, p, **kw):
    d = dict(table=A, width=4, lens=A, n_new=None, group=A, B=2, M=5, H=8, q=A, q_sb=5 * 1024, q_sm=1024, parent=None, out=2 * A, o_sb=5 * 1024,
             o_sm=1024, ws=A, nb=1 << 40)
    d.update(kw)
    return sdv.lib().sd_paged_attn_shared(p, *d.values(), None)


def test_shared_attention_refuses(sdv):
    p = pages(sdv)
    for change, code in [(dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(group=None), EINVAL), (dict(q=None), EINVAL), (dict(out=None), EINVAL),
                         (dict(ws=None), EINVAL), (dict(ws=A + 128), EINVAL), (dict(nb=0), EINVAL), (dict(nb=255), EINVAL), (dict(nb=1 << 12), EINVAL),
                         (dict(width=0), EINVAL), (dict(B=0), EINVAL), (dict(M=0), EINVAL), (dict(H=6), EINVAL), (dict(H=0), EINVAL),
                         (dict(M=17, q_sb=17 * 1024, o_sb=17 * 1024), EUNSUPPORTED), (dict(B=1025), EUNSUPPORTED), (dict(q=A + 4), EINVAL),
                         (dict(q_sm=1022), EINVAL), (dict(o_sm=512), EINVAL), (dict(q_sb=0), EINVAL), (dict(o_sb=0), EINVAL), (dict(width=1 << 28), EUNSUPPORTED)]:
        assert shared(sdv, p, **change) == code, change
    assert shared(sdv, None) == EINVAL and shared(sdv, pages(sdv, D=96)) == EUNSUPPORTED
    for a in ((0, 5, 8, 4, 128), (2, 17, 8, 4, 128), (2, 5, 6, 4, 128), (2, 5, 8, 4, 96), (1025, 5, 8, 4, 128)):
        assert sdv.lib().sd_paged_attn_shared_workspace_bytes(*a) == 0


def draw(sdv, **kw):
    d = dict(logits=A, ld=5000, V=5000, N=3, u=A, T=None, k=None, p=None, low=None, tokens=A, prob=None, probs=None, ldp=0)
    d.update(kw)
    return sdv.lib().sd_sample(*d.values(), None)


def test_sample_refuses(sdv):
    for change, code in [(dict(logits=None), EINVAL), (dict(logits=A + 2), EINVAL), (dict(u=None), EINVAL), (dict(tokens=None), EINVAL), (dict(N=0), EINVAL),
                         (dict(V=0), EINVAL), (dict(ld=4999), EINVAL), (dict(probs=A, ldp=4999), EINVAL), (dict(probs=A + 2, ldp=5000), EINVAL),
                         (dict(V=360449, ld=1 << 20), EUNSUPPORTED), (dict(N=1 << 30), EUNSUPPORTED)]:
        assert draw(sdv, **change) == code, change


def test_outputs_in_the_inputs_place_are_refused(sdv):
    assert shared(sdv, pages(sdv), q=A, out=A) == EINVAL
    assert draw(sdv, logits=A, probs=A, ldp=5000) == EINVAL


def test_python_refuses(sdv):
    import torch
    for kw in (dict(rot=12), dict(rot=0), dict(rot=4)):
        with pytest.raises(sdv.SdError):
            sdv.Rope(**kw)
    with pytest.raises(ValueError):
        sdv.Rope(64, scaling="unknown")
    with pytest.raises(ValueError):
        sdv.Rope(64, inv_freq=[1.0])
    with pytest.raises(sdv.SdError):
        sdv.Rope(64, scaling="yarn", factor=0.5)
    x = torch.zeros(2, 100)
    if not torch.cuda.is_available():
        return
    with pytest.raises(ValueError):
        sdv.sample(x, torch.zeros(2), torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("name,sites", [("sdv_rope.cu", {119, 120, 121, 122}), ("sdv_draw.cu", {123, 124, 125}), ("sdv_paged_shared.cu", {126, 127, 128, 129})])
def test_the_bounds_checked_build_checks_these_kernels(sdv, name, sites):
    import os
    import re
    from speculative_decoding_verify_gb300 import build as b
    assert {int(s) for s in re.findall(r"status,\s*(1\d\d)\)", open(os.path.join(b.CSRC, name)).read())} == sites


def test_a_drawn_token_of_another_place_is_noticed():
    """The check of drawn tokens that the GPU tests use, on rows drawn here with mistakes planted."""
    rng = np.random.default_rng(0)
    for T, k, p, low in ((1.0, 0, 1.0, 0.0), (0.7, 20, 1.0, 0.0), (1.0, 0, 0.8, 0.0), (1.3, 50, 0.9, 0.05), (0.0, 0, 1.0, 0.0)):
        l = (rng.standard_normal(500) * 2).astype(np.float32)
        u = 0.37
        at = plain.order(l.astype(np.float64))
        t, n = (1.0, 1) if T == 0 else (T, k or 500)
        w = np.exp((l.astype(np.float64) - l.max()) / t)
        keep = at[:n]
        run = np.cumsum(w[keep])
        keep = keep[:int((run < p * run[-1]).sum()) + 1] if p < 1 else keep
        keep = keep[w[keep] >= low]
        q = np.zeros(500)
        q[keep] = w[keep] / w[keep].sum()
        token = int((np.cumsum(q) <= u).sum())
        plain.check_row(l, u, T, k, p, low, token, q[token], q)
        plain.check_row(l, u, T, k, p, low, token, q[token], None)
        for wrong in (q[::-1].copy(), np.roll(q, 1)):
            with pytest.raises(AssertionError):
                plain.check_row(l, u, T, k, p, low, token, q[token], wrong)
        if T:
            with pytest.raises(AssertionError):
                plain.check_row(l, u + 0.3, T, k, p, low, token, q[token], q)
            with pytest.raises(AssertionError):
                plain.check_row(l, u, T, k, p, low, token, q[token] * 1.01, None)
