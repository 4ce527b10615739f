"""Promises of the paged cache calls that need no GPU: the header against the
sources, refusals before any CUDA call, the oracle's view of idle requests."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import kv
from speculative_decoding_verification_94_b200 import sv
from tests.test_kv_abi import E, F, U, cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake-pointer validation tests run only without a GPU")


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_94_b200 import build
    build.build()
    return sv.lib()


@no_gpu
def test_commit_ragged_validates(lib):
    def call(c=None, **kw):
        a = dict(layers=2, ls=10 * 16 * 128, B=4, table=F, max_pages=8, kv_len=F, q_len=F, nodes=F,
                 width=6, acc=F, status=None, stream=None)
        a.update(kw)
        return lib.sv_kv_commit_ragged(ctypes.byref(c or cache()), *a.values())
    for kw in (dict(layers=0), dict(ls=-1), dict(ls=9 * 16 * 128), dict(B=-1), dict(table=None),
               dict(kv_len=None), dict(nodes=None), dict(acc=None), dict(max_pages=0),
               dict(width=0), dict(table=F + 2), dict(nodes=F + 2), dict(acc=F + 2),
               dict(q_len=F + 2), dict(status=F + 2)):
        assert call(**kw) == E, kw
    assert call(cache(heads=0)) == E and call(width=1025) == U and call(B=65536) == U
    assert call(B=0) == sv.SV_OK and call(B=0, q_len=None) == sv.SV_OK


def test_a_request_left_out_may_name_another_requests_pages():
    """Why a commit needs q_len: request 0 ends and gives back pages 0 and 1,
    request 1 grows into them, and request 0's table still names them."""
    o = kv.plan([6, 4], [0, 0], [0, 0], [1, 0], [0, 7], [[0, 1, -1], [2, -1, -1]], [2, 1],
                [-1, -1, -1], 0, 4, 7)
    assert o["q_len"].tolist() == [0, 7] and o["block_table"].tolist() == [[0, 1, -1], [2, 1, 0]]
    cache4 = np.arange(3 * 4, dtype=np.float64).reshape(1, 3, 4, 1, 1)
    # verification accepted a path for request 0 too
    moved = kv.commit(cache4, o["block_table"], o["kv_len"], [[0, 2], [0, -1]], [1, 0])
    assert not np.array_equal(moved, cache4)


def _parameters(text, name, end):
    """Parameter names of a function's declaration (end ";") or definition ("{") in C."""
    m = re.search(r"\b%s\s*\(([^()]*(?:\([^()]*\)[^()]*)*)\)\s*%s" % (name, end), text)
    if not m or m.group(1).strip() in ("", "void"):
        return [] if m else None
    return [re.findall(r"\w+", re.sub(r"\[.*?\]", "", p))[-1] for p in m.group(1).split(",")]


def test_the_header_names_its_parameters_as_the_sources_do():
    """A caller reads the prototype: its names are the documented contract
    (a workspace is zeroed, scratch may hold anything)."""
    def plain(path):
        text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
        return re.sub(r"//[^\n]*", "", text)
    header = plain(os.path.join(ROOT, "include", "sv.h"))
    src = os.path.join(ROOT, "speculative_decoding_verification_94_b200", "csrc")
    api = plain(os.path.join(src, "sv_api.cu")), plain(os.path.join(src, "sv_kv.cu"))
    api = "\n".join(t[t.index('extern "C"'):] for t in api)
    short = {"knob_id": "knob", "w": "device_status_word"}  # where the source needs the name itself
    for name in sv.EXPORTS:
        declared, defined = _parameters(header, name, ";"), _parameters(api, name, "{")
        assert declared is not None and defined is not None, name
        assert declared == [short.get(p, p) for p in defined], name


def test_readme_text_positions_of_a_tree_are_places_after_the_commit():
    """The README's lines for the depths of a tree, run on random trees: the
    i-th node of every path from the root stands at kv_len + i, which is where
    a commit of that path puts it, while the plan's positions do not."""
    text = open(os.path.join(ROOT, "README.md")).read()
    block = text[text.index("depth = torch.zeros_like(parents)"):]
    block = block[:block.index("att = ")]
    rng = np.random.default_rng(0)
    n = 24
    par = [[-1] + [int(rng.integers(0, j)) for j in range(1, n)] for _ in range(6)]
    scope = dict(torch=torch, parents=torch.tensor(par, dtype=torch.int32),
                 plan=dict(kv_len=torch.tensor([0, 3, 50, 7, 1, 2], dtype=torch.int32)))
    exec(block, scope)
    got = scope["text_positions"]
    for b, p in enumerate(par):
        base = int(scope["plan"]["kv_len"][b])
        for j in range(n):
            path = kv.ancestors(p, j)[::-1]
            assert got[b, path].tolist() == [base + i for i in range(len(path))]
            # a commit of this path moves node path[i] from place path[i] to place i
            keep = np.arange(base + n, dtype=np.float64).reshape(1, base + n, 1, 1, 1)
            table = [list(range(base + n))]
            moved = kv.commit(keep, table, [base], [path], [len(path) - 1])
            assert [int(moved[0, int(got[b, x]), 0, 0, 0]) - base for x in path] == path
    assert not torch.equal(got, scope["plan"]["kv_len"][:, None] + torch.arange(n))


@no_gpu
def test_tokens_of_more_pieces_than_an_int_counts_are_refused(lib):
    """16-byte to 2-byte pieces of a token, 2^29 to 2^32 of them: refused
    before a count in int can wrap."""
    for heads, d, gap, off in ((1 << 30, 8, 0, 0), (1 << 28, 64, 0, 0), (1 << 26, 128, 0, 0),
                               (1 << 27, 32, 0, 2), (1 << 27, 32, 8, 0), (1 << 27, 33, 0, 0)):
        big = cache(heads=heads, head_dim=d, head_stride=d + gap, token_stride=heads * (d + gap),
                    page_stride=16 * heads * (d + gap), k=F + off, v=F + off)
        ts = heads * d
        pieces = heads * d * 2 // (2 if off or d % 2 else 16)
        got = lib.sv_kv_append(ctypes.byref(big), F, F, 4, 3, 3 * ts, ts, F, None, None)
        assert (got == U) == (pieces > 0x3fffffff), (heads, d)
        got = lib.sv_kv_commit(ctypes.byref(big), 2, 10 * 16 * heads * (d + gap), 4, F, 8, F, F, 6,
                               F, None, None)
        assert (got == U) == (4 * pieces > 0x3fffffff), (heads, d)
    assert lib.sv_kv_commit(ctypes.byref(cache()), 0x7fffffff, 10 * 16 * 128, 4, F, 8, F, F, 6, F,
                            None, None) == U


def test_the_binding_is_rebuilt_for_another_torch(lib, monkeypatch):
    from importlib import metadata

    from speculative_decoding_verification_94_b200 import build
    assert not build._stale()
    version = metadata.version
    monkeypatch.setattr(metadata, "version", lambda name: version(name) + ".other")
    assert build._stale()
