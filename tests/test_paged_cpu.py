"""The calls on a cache in pages refuse what they do not take before anything is launched (no GPU needed)."""
import ctypes

import pytest

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


def attn(sdv, p, **kw):
    d = dict(table=A, width=4, lens=A, n_new=None, B=2, M=5, H=8, q=A, q_sb=5 * 1024, q_sm=1024, parent=None, window=0, sinks=0,
             out=A, o_sb=5 * 1024, o_sm=1024, ws=A, nb=1 << 30)
    d.update(kw)
    return sdv.lib().sd_paged_attn(p, *d.values(), None)


BAD_PAGES = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k=A + 8), EINVAL), (dict(type=3), EUNSUPPORTED), (dict(type=-1), EUNSUPPORTED),
    (dict(n_pages=0), EINVAL), (dict(n_pages=(1 << 30) + 1), EINVAL), (dict(H_kv=0), EINVAL), (dict(page_rows=0), EINVAL), (dict(page_rows=1), EUNSUPPORTED),
    (dict(page_rows=24), EUNSUPPORTED), (dict(page_rows=96, head_stride=96 * 128, page_stride=4 * 96 * 128), EUNSUPPORTED),
    (dict(D=96), EUNSUPPORTED), (dict(D=512), EUNSUPPORTED),
    (dict(row_stride=64), EINVAL), (dict(row_stride=132), EINVAL), (dict(head_stride=128), EINVAL), (dict(page_stride=128), EINVAL),
    (dict(page_stride=-4 * 16 * 128), EINVAL), (dict(type=2, k_scale=None), EINVAL), (dict(type=2, v_scale=A + 4), EINVAL),
]


@pytest.mark.parametrize("change,code", BAD_PAGES)
def test_bad_pages_are_refused_by_every_call(sdv, change, code):
    L, p = sdv.lib(), pages(sdv, **change)
    assert attn(sdv, p) == code
    assert L.sd_paged_append(p, A, 4, A, None, 2, 5, A, A, 5 * 512, 512, None) == code
    assert L.sd_paged_commit(p, A, 4, A, 2, 5, None, A, None) == code
    assert L.sd_pages_reserve(p, A, A, 4, A, None, 2, 5, A, A, 1 << 30, None) == code
    assert L.sd_pages_copy(p, A, 1 << 30, None) == code
    assert L.sd_pages_compact(p, A, A, 4, 2, A, A, A, 1 << 30, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(width=0), EINVAL), (dict(B=0), EINVAL), (dict(M=0), EINVAL), (dict(H=6), EINVAL), (dict(H=2), EINVAL), (dict(H=0), EINVAL),
    (dict(window=-1), EINVAL), (dict(sinks=-1), EINVAL), (dict(M=17, q_sb=17 * 1024, o_sb=17 * 1024), EUNSUPPORTED),
    (dict(B=1025), EUNSUPPORTED), (dict(q=A + 4), EINVAL), (dict(out=A + 8), EINVAL), (dict(ws=A + 128), EINVAL),
    (dict(q_sm=1022), EINVAL), (dict(q_sm=1025), EINVAL), (dict(o_sm=512), EINVAL), (dict(q_sb=0), EINVAL), (dict(o_sb=0), EINVAL),
    (dict(width=1 << 28), EUNSUPPORTED),
])
def test_attention_refuses(sdv, change, code):
    assert attn(sdv, pages(sdv), **change) == code


def test_append_and_commit_refuse(sdv):
    L, p = sdv.lib(), pages(sdv)
    ok = dict(table=A, width=4, lens=A, n_new=None, B=2, M=5, k=A, v=A, sb=5 * 512, sm=512)
    for change, code in [(dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(k=None), EINVAL), (dict(v=A + 4), EINVAL),
                         (dict(B=0), EINVAL), (dict(M=0), EINVAL), (dict(sm=511), EINVAL), (dict(sm=514), EINVAL), (dict(sb=0), EINVAL),
                         (dict(width=0), EINVAL), (dict(B=1025), EUNSUPPORTED), (dict(width=1 << 28), EUNSUPPORTED)]:
        assert L.sd_paged_append(p, *{**ok, **change}.values(), None) == code, change
    ok = dict(table=A, width=4, lens=A, B=2, M=5, path=A, count=A)
    for change, code in [(dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(count=None), EINVAL), (dict(M=0), EINVAL),
                         (dict(M=17), EUNSUPPORTED), (dict(B=1025), EUNSUPPORTED), (dict(B=0), EINVAL)]:
        assert L.sd_paged_commit(p, *{**ok, **change}.values(), None) == code, change


def test_page_calls_refuse(sdv):
    L, p = sdv.lib(), pages(sdv)
    need = L.sd_pages_workspace_bytes(10, 2, 4)
    assert need > 0 and L.sd_pages_workspace_bytes(0, 2, 4) == 0 and L.sd_pages_workspace_bytes(10, 0, 4) == 0
    ok = dict(refs=A, table=A, width=4, lens=A, n_new=None, B=2, M=5, missing=A, ws=A, nb=need)
    for change in (dict(refs=None), dict(table=None), dict(lens=None), dict(missing=None), dict(ws=None), dict(ws=A + 16), dict(nb=need - 1),
                   dict(M=0), dict(B=0), dict(width=0)):
        assert L.sd_pages_reserve(p, *{**ok, **change}.values(), None) == EINVAL, change
    assert L.sd_pages_reserve(p, *{**ok, **dict(B=1025, nb=1 << 40)}.values(), None) == EUNSUPPORTED
    ok = dict(refs=A, table=A, width=4, B=2, remap=A, n_live=A, ws=A, nb=need)
    for change in (dict(refs=None), dict(table=None), dict(remap=None), dict(n_live=None), dict(ws=None), dict(nb=need - 1), dict(B=0)):
        assert L.sd_pages_compact(p, *{**ok, **change}.values(), None) == EINVAL, change
    ok = dict(refs=A, n=10, table=A, width=4, lens=A, B=4, P=16, src=A, dst=A, k=3)
    for change in (dict(refs=None), dict(n=0), dict(table=None), dict(lens=None), dict(src=None), dict(dst=None), dict(k=-1), dict(k=5), dict(P=0)):
        assert L.sd_pages_fork(*{**ok, **change}.values(), None) == EINVAL, change
    assert L.sd_pages_fork(*{**ok, **dict(k=0)}.values(), None) == 0
    ok = dict(refs=A, n=10, table=A, width=4, lens=A, B=4, P=16, seqs=A, keep=None, k=3)
    for change in (dict(refs=None), dict(table=None), dict(seqs=None), dict(k=-1), dict(B=0)):
        assert L.sd_pages_free(*{**ok, **change}.values(), None) == EINVAL, change
    ok = dict(refs=A, n=10, table=A, width=4, lens=A, B=4, P=16, window=8, sinks=0)
    for change in (dict(refs=None), dict(table=None), dict(lens=None), dict(window=0), dict(sinks=-1), dict(P=0)):
        assert L.sd_pages_trim(*{**ok, **change}.values(), None) == EINVAL, change


def test_workspace_sizes_of_refused_shapes_are_zero(sdv):
    L = sdv.lib()
    for a in ((0, 5, 8, 4, 128), (2, 17, 8, 4, 128), (2, 5, 6, 4, 128), (2, 5, 8, 4, 96), (1025, 5, 8, 4, 128)):
        assert L.sd_paged_attn_workspace_bytes(*a) == 0


def test_python_refuses_tensors_that_are_not_on_the_gpu(sdv):
    import torch
    with pytest.raises(ValueError):
        sdv.KvPages(torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 16, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        sdv.KvPages(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64))


@pytest.mark.parametrize("name", ["sdv_pages.cu", "sdv_paged_attn.cuh", "sdv_paged_attn.cu", "sdv_paged_wide.cuh"])
def test_the_bounds_checked_build_checks_the_paged_kernels(sdv, name):
    """Each file with paged kernels has its sites (109 to 118), which the bounds-checked suite runs."""
    import os
    import re
    from speculative_decoding_verify_gb300 import build as b
    text = open(os.path.join(b.CSRC, name)).read()
    sites = {int(s) for s in re.findall(r"status,\s*(1\d\d)\)", text)}
    assert sites and sites <= set(range(109, 119))
