"""Refusals of the paged cache calls: bad arguments return before any CUDA
call (so these run without a GPU), and the binding refuses what the C call
could not see."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_94_b200 import sv

F = 0x10000  # never dereferenced
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake-pointer validation tests run only without a GPU")
E, U, W = sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED, sv.SV_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_94_b200 import build
    build.build()
    return sv.lib()


def cache(**kw):
    a = dict(k=F, v=F, dtype=sv.SV_BF16, num_pages=10, page_size=16, heads=2, head_dim=64,
             page_stride=16 * 128, token_stride=128, head_stride=64)
    a.update(kw)
    return sv.sv_kv_cache(*a.values())


BAD_CACHES = [
    dict(k=None), dict(v=None), dict(dtype=5), dict(num_pages=0), dict(page_size=0), dict(heads=0),
    dict(head_dim=0), dict(k=F + 1), dict(v=F + 1), dict(head_stride=-64),
    dict(head_stride=63),                      # heads overlap
    dict(token_stride=64),                     # a token's heads overlap the next token
    dict(page_stride=15 * 128),                # pages overlap
    dict(page_stride=0),
]


def _plan(lib, **kw):
    a = dict(kv_len=F, written=F, acc=F, rel=F, new=F, B=4, max_new=4, page=16, num_pages=100,
             table=F, max_pages=10, pages=F, free=F, count=F, kv_out=F, pages_out=F, count_out=F,
             q_len=F, slots=F, pos=F, status=F, stream=None)
    a.update(kw)
    return lib.sv_kv_plan(*a.values())


@no_gpu
def test_plan_validates(lib):
    for name in ("kv_len", "new", "table", "pages", "free", "count", "kv_out", "pages_out",
                 "count_out", "q_len", "slots"):
        assert _plan(lib, **{name: None}) == E, name
        assert _plan(lib, **{name: F + 2}) == E, name
    for name in ("written", "acc", "rel", "pos", "status"):
        assert _plan(lib, **{name: F + 2}) == E, name
    assert _plan(lib, slots=F + 4) == E                    # int64
    assert _plan(lib, written=None) == E                   # accepted_len needs it
    for name in ("max_new", "page", "num_pages", "max_pages"):
        assert _plan(lib, **{name: 0}) == E, name
    assert _plan(lib, B=-1) == E
    assert _plan(lib, B=8193) == U
    assert _plan(lib, B=8192, max_pages=1 << 18) == U
    assert _plan(lib, B=8192, max_new=1 << 18) == U
    assert _plan(lib, B=0) == sv.SV_OK
    assert _plan(lib, B=0, count=None) == E


@no_gpu
def test_append_validates(lib):
    def call(c=None, k=F, v=F, B=4, n=3, bs=384, ts=128, slots=F, status=None):
        return lib.sv_kv_append(ctypes.byref(c or cache()), k, v, B, n, bs, ts, slots, status, None)
    for kw in BAD_CACHES:
        assert call(cache(**kw)) == E, kw
    assert call(cache(head_dim=257, head_stride=257, token_stride=514, page_stride=16 * 514)) == U
    assert lib.sv_kv_append(None, F, F, 4, 3, 384, 128, F, None, None) == E
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(k=F + 1), dict(slots=F + 4),
               dict(B=-1), dict(n=0), dict(bs=-1), dict(ts=-1), dict(status=F + 1)):
        assert call(**kw) == E, kw
    assert call(B=0) == sv.SV_OK


@no_gpu
def test_attend_validates(lib):
    big = 1 << 30

    def call(c=None, **kw):
        a = dict(q=F, bs=1024, ts=256, B=4, n=4, hq=4, table=F, max_pages=8, kv_len=F, q_len=F,
                 parents=F, scale=0.125, out=F + 4096, lse=F, ws=F, wsb=big, status=None,
                 stream=None)
        a.update(kw)
        return lib.sv_kv_attend(ctypes.byref(c or cache()), *a.values())
    for kw in BAD_CACHES:
        assert call(cache(**kw)) == E, kw
    for kw in (dict(q=None), dict(out=None), dict(table=None), dict(kv_len=None), dict(q=F + 1),
               dict(out=F + 1), dict(table=F + 2), dict(kv_len=F + 2), dict(q_len=F + 2),
               dict(parents=F + 2), dict(lse=F + 2), dict(status=F + 2), dict(B=-1), dict(n=0),
               dict(n=1025), dict(hq=0), dict(hq=3), dict(max_pages=0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38),
               dict(bs=-1), dict(ts=-1), dict(out=F)):
        assert call(**kw) == E, kw
    assert call(hq=1 << 17) == U
    need = lib.sv_kv_attend_scratch_size(4, 4, 4, 2, 64, sv.SV_BF16)
    assert need > 0
    assert call(ws=None) == W and call(ws=F + 8) == W and call(wsb=need - 1) == W
    assert call(B=0, ws=None) == sv.SV_OK
    assert lib.sv_kv_attend_scratch_size(4, 4, 4, 2, 257, sv.SV_BF16) == 0
    assert lib.sv_kv_attend_scratch_size(4, 0, 4, 2, 64, sv.SV_BF16) == 0


@no_gpu
def test_commit_validates(lib):
    def call(c=None, **kw):
        a = dict(layers=2, ls=10 * 16 * 128, B=4, table=F, max_pages=8, kv_len=F, nodes=F, width=6,
                 acc=F, status=None, stream=None)
        a.update(kw)
        return lib.sv_kv_commit(ctypes.byref(c or cache()), *a.values())
    for kw in BAD_CACHES:
        assert call(cache(**kw)) == E, kw
    for kw in (dict(layers=0), dict(ls=-1), dict(ls=9 * 16 * 128), dict(B=-1), dict(table=None),
               dict(kv_len=None), dict(nodes=None), dict(acc=None), dict(max_pages=0),
               dict(width=0), dict(table=F + 2), dict(nodes=F + 2), dict(acc=F + 2)):
        assert call(**kw) == E, kw
    assert call(width=1025) == U and call(B=65536) == U
    assert call(B=0) == sv.SV_OK


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    c = torch.zeros(3, 4, 1, 8, dtype=torch.bfloat16)
    x = torch.zeros(2, 1, 1, 8, dtype=torch.bfloat16)
    for call in (lambda: sv.sv_kv_plan(i, t, i, i, i[:1], i, 1, 4),
                 lambda: sv.sv_kv_append(x, x, torch.zeros(2, 1, dtype=torch.int64), c, c),
                 lambda: sv.sv_kv_attend(x, c, c, t, i),
                 lambda: sv.sv_kv_commit(c, c, t, i, t, i)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
