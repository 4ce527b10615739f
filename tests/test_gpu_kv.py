"""The paged cache calls on the GPU against the float64 oracle."""
import random

import numpy as np
import pytest
import torch

from oracle import kv as O
from speculative_decoding_verification_94_b200 import sv
from tests.test_kv_oracle import random_plan

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def run_plan(args, page, mx, in_place=False, positions=True):
    kv_len, written, acc, rel, new, table, pages, free, count = args
    t = dict(kv_len=i32(kv_len), new=i32(new), pages=i32(pages), count=i32([count]),
             table=i32(table), free=i32(free))
    st = status()
    out = dict(kv_len=t["kv_len"], pages=t["pages"], free_count=t["count"],
               q_len=t["new"]) if in_place else None
    o = sv.sv_kv_plan(t["kv_len"], t["table"], t["pages"], t["free"], t["count"], t["new"], mx,
                      page, written=None if written is None else i32(written),
                      accepted_len=None if acc is None else i32(acc),
                      release=None if rel is None else i32(rel), out=out, device_status=st)
    got = {k: v.cpu().numpy() for k, v in o.items()}
    got["block_table"], got["free_pages"] = t["table"].cpu().numpy(), t["free"].cpu().numpy()
    return got, int(st.item())


def check_plan(got, ref):
    for k in ("kv_len", "pages", "q_len", "slot_map", "positions", "block_table", "free_pages"):
        assert np.array_equal(got[k], ref[k]), k
    assert int(got["free_count"][0]) == ref["free_count"]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,max_pages,mx,extra", [
    (1, 16, 4, 1, 3), (1, 1, 40, 5, 50), (7, 3, 30, 9, 0), (32, 16, 20, 4, 8), (33, 16, 40, 8, 500),
    (100, 7, 20, 32, 10), (1100, 16, 12, 4, 900), (2500, 4, 16, 3, 100), (8192, 16, 3, 1, 4000),
    (40, 16, 70, 500, 1200), (6, 16, 300, 4097, 200), (3, 5, 2100, 10001, 6100)])
def test_plan_matches_the_oracle(B, page, max_pages, mx, extra, in_place):
    rng = random.Random(B * 31 + mx)
    args = random_plan(rng, B, page, max_pages, mx, extra)
    got, st = run_plan(args, page, mx, in_place)
    ref = O.plan(*args, page, mx)
    check_plan(got, ref)
    assert st == (sv.SV_DEV_NO_PAGES if ref["starved"] else 0)


def test_plan_optional_inputs():
    rng = random.Random(5)
    a = list(random_plan(rng, 20, 16, 20, 6, 100, release=0.0))
    for written, acc, rel in ((None, None, None), (a[1], None, None), (a[1], None, a[3])):
        b = list(a)
        b[1], b[2], b[3] = written, acc, rel
        if written is None:
            b[6] = [-(-x // 16) for x in b[0]]
            b[5] = [r[:n] + [-7] * (20 - n) for r, n in zip(b[5], b[6])]
        got, st = run_plan(b, 16, 6)
        check_plan(got, O.plan(*b, 16, 6))
        assert st == 0


def test_plan_fails_only_the_requests_with_bad_lengths():
    # request 0 is sound; the others break one rule each
    kv_len = [10, -1, 10, 10, 10, 62, 30, 10]
    written = [2, 0, -1, 2, 2, 1, 1, 2]
    acc = [1, -1, -1, 2, 1, 0, 0, 1]           # 3: accepted >= written
    new = [3, 1, 1, 1, 9, 2, 1, -2]            # 4: new > max_new; 5: past the table; 7: < 0
    pages = [1, 1, 1, 1, 1, 4, 1, 1]           # 6: 31 tokens on one page
    table = [[b, 20 + b, 40 + b, 60 + b] for b in range(8)]
    free = list(range(80, 90)) + [-1] * 80
    args = (kv_len, written, acc, None, new, table, pages, free, 10)
    got, st = run_plan(args, 16, 8)
    assert st == sv.SV_DEV_BAD_LEN
    assert got["kv_len"].tolist() == [12] + kv_len[1:]
    assert got["pages"].tolist() == pages and got["q_len"].tolist() == [3] + [0] * 7
    assert got["slot_map"][0].tolist() == [12, 13, 14] + [-1] * 5
    assert (got["slot_map"][1:] == -1).all() and (got["positions"][1:] == -1).all()
    assert int(got["free_count"][0]) == 10
    assert np.array_equal(got["block_table"], np.array(table))


def test_plan_bad_pages_and_counts():
    # a bad page id on the stack: its slots are -1
    args = ([16], None, None, None, [2], [[3, -5]], [1], [0, 1, 99, 7], 3)
    got, st = run_plan(args, 16, 2)
    assert st == sv.SV_DEV_BAD_INDEX and (got["slot_map"] == -1).all()
    # a stack that claims more than it can hold
    got, st = run_plan(([16], None, None, None, [2], [[3, -5]], [1], [0, 1, 2, 3], 9), 16, 2)
    assert st & sv.SV_DEV_BAD_LEN and got["slot_map"].tolist() == [[48, 49]]
    got, st = run_plan(([16], None, None, None, [2], [[3, -5]], [1], [0, 1, 2, 3], -2), 16, 2)
    assert st == sv.SV_DEV_BAD_LEN | sv.SV_DEV_NO_PAGES and (got["slot_map"] == -1).all()
    # pages given back twice do not run past the stack's end
    got, st = run_plan(([40], None, None, [1], [0], [[1, 2, 3]], [3], [5, 6, 7, 8], 3), 16, 2)
    assert st == sv.SV_DEV_BAD_LEN and got["free_pages"].tolist() == [5, 6, 7, 1]
    assert int(got["free_count"][0]) == 4


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def make_cache(pages, page, heads, d, dtype, layout, seed, fill=None):
    """k and v caches [pages, page, heads, d] in several memory layouts."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape):
        if fill is not None:
            return torch.full(shape, fill, dtype=dtype, device=DEV)
        return torch.randn(shape, generator=g, device=DEV).to(dtype)
    if layout == "dense":
        return rnd(pages, page, heads, d), rnd(pages, page, heads, d)
    if layout == "heads_first":
        return tuple(rnd(pages, heads, page, d).transpose(1, 2) for _ in range(2))
    if layout == "joint":  # keys and values of a page in one block
        t = rnd(pages, 2, page, heads, d)
        return t[:, 0], t[:, 1]
    if layout == "padded":  # rows that no 16-byte access fits
        t = rnd(2, pages, page, heads, d + 3)
        return t[0, ..., 1:d + 1], t[1, ..., 1:d + 1]
    raise ValueError(layout)


LAYOUTS = ["dense", "heads_first", "joint", "padded"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,n,heads,d,page,dtype,cut", [
    (1, 1, 1, 1, 1, "f32", 0), (3, 4, 2, 64, 16, "bf16", 0), (5, 33, 4, 128, 16, "bf16", 2),
    (2, 100, 3, 40, 7, "bf16", 1), (4, 9, 2, 6, 5, "bf16", 1), (300, 2, 1, 256, 128, "f32", 3),
    (2, 700, 8, 64, 64, "f32", 1)])
def test_append_writes_its_slots_and_nothing_else(B, n, heads, d, page, dtype, cut, layout):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pages = -(-B * n // page) + 3
    kc, vc = make_cache(pages, page, heads, d, dt, layout, 1)
    g = torch.Generator().manual_seed(B * n)
    slots = torch.randperm(pages * page, generator=g)[:B * n].reshape(B, n)
    slots[torch.rand(B, n, generator=g) < 0.2] = -1
    # parts of one projection output: strided tokens, `cut` leading heads skipped
    x = torch.randn(B, n, cut + 2 * heads, d, generator=g).to(dt).to(DEV)
    k, v = x[:, :, cut:cut + heads], x[:, :, cut + heads:]
    want_k, want_v = kc.clone(), vc.clone()
    for b in range(B):
        for i in range(n):
            s = int(slots[b, i])
            if s >= 0:
                want_k[s // page, s % page] = k[b, i]
                want_v[s // page, s % page] = v[b, i]
    st = status()
    sv.sv_kv_append(k, v, slots.to(DEV), kc, vc, device_status=st)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and int(st.item()) == 0


def test_append_skips_slots_outside_the_cache():
    kc, vc = make_cache(2, 4, 1, 8, torch.float32, "dense", 1)
    before = kc.clone(), vc.clone()
    k = torch.randn(1, 3, 1, 8, device=DEV)
    st = status()
    slots = torch.tensor([[8, 1 << 40, -(1 << 40)]], device=DEV)
    sv.sv_kv_append(k, k, slots, kc, vc, device_status=st)
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    assert int(st.item()) == sv.SV_DEV_BAD_INDEX


# ---------------------------------------------------------------------------
# attend
# ---------------------------------------------------------------------------
def random_tree(rng, n):
    return [-1] + [rng.randint(max(-1, j - 9), j - 1) for j in range(1, n)]


def scenario(B, n, hq, hkv, d, page, lens, dtype, *, tree=False, ragged=False, layout="dense",
             seed=0, q_scale=2.0, spare=3):
    rng = random.Random(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kv_len = [lens[b % len(lens)] for b in range(B)]
    q_len = [n if not ragged else rng.choice([0, n, rng.randint(0, n)]) for _ in range(B)]
    cnt = [-(-(a + m) // page) for a, m in zip(kv_len, q_len)]
    total = sum(cnt) + spare
    ids = list(range(total))
    rng.shuffle(ids)
    mp = max(max(cnt), 1) + 1
    table, at = [], 0
    for b in range(B):
        table.append(ids[at:at + cnt[b]] + [-3] * (mp - cnt[b]))
        at += cnt[b]
    kc, vc = make_cache(total, page, hkv, d, dt, layout, seed + 1)
    g = torch.Generator(device=DEV).manual_seed(seed + 2)
    q = (q_scale * torch.randn(B, n, hq, d, generator=g, device=DEV)).to(dt)
    par = [random_tree(rng, n) for _ in range(B)] if tree else None
    return dict(q=q, kc=kc, vc=vc, table=table, kv_len=kv_len, q_len=q_len, parents=par,
                scale=d ** -0.5, page=page)


def call_attend(s, **kw):
    st = status()
    o = sv.sv_kv_attend(s["q"], s["kc"], s["vc"], i32(s["table"]), i32(s["kv_len"]),
                        q_len=i32(s["q_len"]), parents=None if s["parents"] is None else
                        i32(s["parents"]), scale=s["scale"], device_status=st, **kw)
    return o["out"], o["lse"], int(st.item())


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_attend(s, out, lse, rows=None):
    """Against the oracle.  eps = 2^-24 is half a step of fp32.  A score is
    off by at most (d + 4) eps size (d products summed, scale and log2 e
    rounded), a weight by that much more relatively, 3 eps for its power of
    two, the same again for the rescaling of each 16-key part by which the
    maximum can grow; sums of N terms add N eps.  Numerator and denominator
    both have these errors (factor 2).  bf16 weights enter the numerator only:
    as a sum of two bf16 they are off by 2^-16 up to 16 rows a key head, as
    one bf16 by half a step, 2^-8, beyond (sum |dp v| <= 2^-8 sum p |v|).  fp32
    products of more than 8 rows go through two-part tf32 and are off by 20 eps
    each: 20 eps size of a score and 20 eps of the numerator, counted for both
    types.  The output then rounds
    by half a step of its type."""
    ref, rl, size, absv = O.attend(host(s["q"]), host(s["kc"]), host(s["vc"]), s["table"],
                                   s["kv_len"], s["q_len"], s["parents"], s["scale"])
    d = s["q"].shape[-1]
    eps = 2.0 ** -24
    bf = s["q"].dtype == torch.bfloat16
    n_keys = np.array(s["kv_len"])[:, None, None] + s["q"].shape[1]
    w = ((2 * (d + 4) + 20) * size + n_keys + 6 * (n_keys / 16 + 2)) * eps
    rows = s["q"].shape[1] * s["q"].shape[2] // s["kc"].shape[2]
    rel = 2 * w + 20 * eps + (0.0 if not bf else 2.0 ** -16 if rows <= 16 else 2.0 ** -8)
    tol = rel[..., None] * absv + (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(ref) + 1e-37
    got, gl = host(out), lse.cpu().numpy().astype(np.float64)
    for b in range(got.shape[0]):
        m = s["q_len"][b]
        assert (np.abs(got[b, :m] - ref[b, :m]) <= tol[b, :m]).all(), (
            b, np.nanmax(np.abs(got[b, :m] - ref[b, :m]) / tol[b, :m]))
        assert (got[b, m:] == 0).all() and (gl[b, m:] == -np.inf).all()
        lt = w[b, :m] + 4 * eps * (1 + np.abs(rl[b, :m]))
        assert (np.abs(gl[b, :m] - rl[b, :m]) <= lt).all()


CASES = [
    # B, n, hq, hkv, d, page, lens
    (1, 1, 1, 1, 64, 16, [0]),              # the first token of a request
    (1, 1, 8, 1, 128, 16, [1]),
    (3, 1, 28, 4, 128, 16, [15, 16, 17]),   # around a page's end
    (4, 1, 8, 8, 64, 1, [5, 63, 64, 65]),   # pages of one token, no sharing of heads
    (2, 4, 14, 2, 128, 16, [127, 300]),     # 28 rows
    (2, 5, 10, 2, 128, 3, [31, 200]),       # 25 rows, odd pages
    (3, 8, 8, 2, 64, 32, [0, 7, 500]),      # 32 rows
    (2, 8, 10, 2, 128, 16, [100, 259]),     # 40 rows
    (2, 16, 16, 2, 128, 128, [90, 401]),    # 128 rows
    (1, 33, 8, 1, 64, 64, [130]),           # 264 rows
    (1, 32, 16, 2, 128, 32, [700]),         # 256 rows
    (2, 3, 6, 2, 80, 24, [50, 77]),         # head sizes that are not a power of two
    (2, 2, 4, 2, 96, 16, [50, 77]),
    (2, 2, 4, 2, 256, 16, [50, 77]),
    (1, 2, 3, 1, 7, 5, [50]),
    (1, 1, 2, 1, 1, 2, [9]),
    (1, 1, 4, 1, 128, 16, [6000]),          # split over many blocks
    (1, 7, 8, 1, 128, 16, [5003]),
    (1, 12, 8, 1, 64, 16, [5003]),
    (200, 1, 2, 1, 64, 16, [0, 1, 40, 90]),  # more requests than threads of a warp
    (700, 1, 1, 1, 64, 16, [3, 0, 17]),      # more requests than threads of a block
    (2, 20, 16, 2, 128, 24, [100, 259]),    # 160 rows, pages that no tile is a multiple of
    (2, 20, 16, 2, 64, 4, [100, 259]),      # and pages too small for a tile's boxes
    (2, 9, 8, 2, 128, 8, [100, 259]),       # 36 rows, the smallest pages that boxes take
    (2, 20, 16, 2, 128, 256, [100, 700]),   # pages larger than a tile
    (2, 3, 8, 2, 40, 16, [33, 300]),        # head sizes inside a kernel's 64 or 128 columns
    (2, 20, 8, 2, 40, 16, [33, 300]),
    (2, 9, 8, 2, 112, 16, [33, 700]),
    (2, 40, 8, 2, 72, 32, [33, 300]),
    (2, 4, 8, 2, 8, 16, [33, 300]),
    (2, 12, 8, 2, 8, 16, [33, 300]),
    (2, 12, 8, 2, 100, 16, [33, 300]),      # 16-byte rows in fp32 only
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,hq,hkv,d,page,lens", CASES)
def test_attend_chain(B, n, hq, hkv, d, page, lens, dtype):
    s = scenario(B, n, hq, hkv, d, page, lens, dtype, seed=n * 7 + d)
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,hq,hkv,d,page,lens", [c for c in CASES if c[1] > 1])
def test_attend_tree_and_ragged(B, n, hq, hkv, d, page, lens, dtype):
    s = scenario(B + 2, n, hq, hkv, d, page, lens, dtype, tree=True, ragged=True, seed=n + d)
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


@pytest.mark.parametrize("layout", LAYOUTS[1:])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", [(1, 4), (4, 12), (20, 8)])
def test_attend_layouts(layout, dtype, n, hq):
    s = scenario(3, n, hq, 2, 64, 16, [3, 70, 200], dtype, ragged=True, layout=layout, seed=9)
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


@pytest.mark.parametrize("n,g", [(1, 4), (4, 7), (16, 8)])
def test_attend_query_inside_a_projection(n, g):
    s = scenario(3, n, 2 * g, 2, 128, 16, [3, 70, 200], "bf16", ragged=True, seed=9)
    fused = torch.randn(3, n, 2 * g + 4, 128, device=DEV).bfloat16()
    fused[:, :, :2 * g] = s["q"]
    dense = call_attend(s)
    s["q"] = fused[:, :, :2 * g]
    out, lse, st = call_attend(s)
    assert st == 0 and torch.equal(out, dense[0]) and torch.equal(lse, dense[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 48])
@pytest.mark.parametrize("n,hq,tree", [(1, 4, False), (5, 4, False), (5, 4, True), (9, 12, True),
                                       (40, 8, True)])
def test_attend_ignores_what_it_does_not_attend_to(n, hq, d, tree, dtype):
    """NaN, infinities and the type's lowest value in every place a row does
    not attend to: free pages, the rest of the last page, later tokens of a
    chain, other branches of a tree."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    s = scenario(3, n, hq, 2, d, 16, [0, 5, 77], dtype, tree=tree, seed=21)
    clean = call_attend(s)
    bad = [float("nan"), float("inf"), -float("inf"), torch.finfo(dt).min]
    used = torch.zeros(s["kc"].shape[:2], dtype=torch.bool)
    for b in range(3):
        for t in range(s["kv_len"][b] + s["q_len"][b]):
            used[s["table"][b][t // 16], t % 16] = True
    free = (~used).to(DEV)
    for j, c in enumerate((s["kc"], s["vc"])):
        c[free] = torch.tensor(bad[j], device=DEV).to(dt)
    out, lse, st = call_attend(s)
    assert st == 0 and torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    # the last new token of each request: only rows that see it may change
    if n > 1:
        for val in bad:
            t = dict(s, kc=s["kc"].clone(), vc=s["vc"].clone())
            for b in range(3):
                at = s["kv_len"][b] + n - 1
                t["kc"][s["table"][b][at // 16], at % 16] = val
                t["vc"][s["table"][b][at // 16], at % 16, :, ::2] = val
            o2, l2, st = call_attend(t)
            assert st == 0
            assert torch.equal(o2[:, :-1], clean[0][:, :-1])
            assert torch.equal(l2[:, :-1], clean[1][:, :-1])


@pytest.mark.parametrize("n,hq", [(2, 4), (6, 12), (20, 16)])
def test_attend_infinite_values_reach_the_rows_that_see_them(n, hq):
    s = scenario(2, n, hq, 2, 128, 16, [3, 90], "bf16", seed=5)
    t = dict(s, vc=s["vc"].clone())
    for b in range(2):
        at = s["kv_len"][b] + 1  # seen by tokens 1, 2, ...
        t["vc"][s["table"][b][at // 16], at % 16, :, 3] = float("inf")
        t["vc"][s["table"][b][at // 16], at % 16, :, 8] = float("nan")
    clean, out = call_attend(s)[0], call_attend(t)[0]
    keep = [c for c in range(128) if c not in (3, 8)]
    assert torch.equal(out[:, 0], clean[:, 0])
    assert torch.equal(out[..., keep], clean[..., keep])
    assert torch.isinf(out[:, 1:, :, 3]).all() and torch.isnan(out[:, 1:, :, 8]).all()


@pytest.mark.parametrize("n,hq,dtype", [(6, 4, "bf16"), (20, 16, "bf16"), (40, 8, "bf16"),
                                        (6, 4, "f32"), (20, 16, "f32")])
def test_attend_bad_parents_beside_infinite_values(n, hq, dtype):
    """Walks up a tree end at a bad parent, in the search for values that are
    not finite too."""
    s = scenario(3, n, hq, 2, 128, 16, [40, 3, 90], dtype, tree=True, seed=8)
    t = dict(s, parents=[list(r) for r in s["parents"]], vc=s["vc"].clone())
    t["parents"][0][n - 1] = n - 1          # itself
    t["parents"][0][n - 2] = n - 1          # each other
    t["parents"][1][n - 1] = n + 5          # no node
    t["parents"][1][n - 2] = -7
    for b in range(3):
        at = s["kv_len"][b]
        t["vc"][s["table"][b][at // 16], at % 16, :, 5] = float("inf")
    out, lse, st = call_attend(t)
    assert st == sv.SV_DEV_BAD_TREE
    for b in range(2):
        assert torch.isnan(out[b, n - 2:]).all() and torch.isnan(lse[b, n - 2:]).all()
    # the sound request: infinite where the root is an ancestor
    clean = call_attend(s)[0]
    keep = [c for c in range(128) if c != 5]
    assert torch.equal(out[2][..., keep], clean[2][..., keep])
    for i in range(n):
        root = 0 in O.ancestors(s["parents"][2], i)
        assert bool(torch.isinf(out[2, i, :, 5]).all()) == root


@pytest.mark.parametrize("n,hq,d", [(1, 4, 128), (8, 8, 64), (20, 8, 128), (3, 4, 40)])
def test_attend_bad_inputs_fail_only_their_rows(n, hq, d):
    s = scenario(4, n, hq, 2, d, 16, [40, 40, 40, 40], "bf16", tree=True, seed=3)
    clean = call_attend(s)[0]
    t = dict(s, table=[list(r) for r in s["table"]], kv_len=list(s["kv_len"]))
    t["table"][1][1] = 10 ** 6
    out, lse, st = call_attend(t)
    assert st == sv.SV_DEV_BAD_INDEX and torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])
    t = dict(s, kv_len=[40, 40, -1, 40])
    out, lse, st = call_attend(t)
    assert st == sv.SV_DEV_BAD_LEN and torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()
    t = dict(s, kv_len=[40, 40, 10 ** 6, 40], q_len=[n, n, n, n + 1])
    out, lse, st = call_attend(t)
    assert st == sv.SV_DEV_BAD_LEN and torch.isnan(out[2:]).all()
    if n > 1:
        t = dict(s, parents=[list(r) for r in s["parents"]])
        t["parents"][3][n - 1] = n - 1  # its own parent
        out, lse, st = call_attend(t)
        assert st == sv.SV_DEV_BAD_TREE and torch.isnan(out[3, n - 1]).all()
        assert torch.isfinite(out[:3].float()).all()


@pytest.mark.parametrize("n,hq,dtype", [(1, 4, "bf16"), (3, 14, "bf16"), (10, 16, "bf16"),
                                        (40, 8, "bf16"), (2, 8, "f32")])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 4.0])
def test_attend_scales(n, hq, dtype, scale):
    s = scenario(2, n, hq, 2, 64, 16, [33, 200], dtype, tree=True, seed=13, q_scale=0.5)
    s["scale"] = scale
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


@pytest.mark.parametrize("n,g", [(1, 3), (3, 7), (9, 4), (20, 8)])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_attend_queries_off_16_bytes(n, g, shift):
    s = scenario(2, n, 2 * g, 2, 128, 16, [20, 300], "bf16", seed=17)
    buf = torch.empty(s["q"].numel() + shift, dtype=torch.bfloat16, device=DEV)
    q = buf[shift:].view(s["q"].shape)
    q.copy_(s["q"])
    s["q"] = q
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


@pytest.mark.parametrize("n,hq,dtype", [(1, 4, "bf16"), (3, 14, "bf16"), (20, 16, "bf16"),
                                        (4, 8, "f32")])
def test_attend_a_batch_that_is_idle_but_for_a_few(n, hq, dtype):
    s = scenario(300, n, hq, 2, 64, 16, [5, 90, 40], dtype, seed=19)
    s["q_len"] = [n if b in (0, 7, 150, 298) else 0 for b in range(300)]
    s["kv_len"] = [x if m else -5 for x, m in zip(s["kv_len"], s["q_len"])]  # not looked at
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


@pytest.mark.parametrize("n,hq", [(1, 4), (20, 4)])
def test_attend_finds_one_bad_page_among_many(n, hq):
    """More pages than a block looks at in one go."""
    num = 90000
    g = torch.Generator(device=DEV).manual_seed(0)
    k = torch.randn(num, 8, 1, 64, generator=g, device=DEV).bfloat16()
    v = torch.randn(num, 8, 1, 64, generator=g, device=DEV).bfloat16()
    q = torch.randn(1, n, hq, 64, generator=g, device=DEV).bfloat16()
    table = torch.randperm(num, generator=g, device=DEV).int()[None].contiguous()
    kv_len = i32([num * 8 - n])
    st = status()
    o = sv.sv_kv_attend(q, k, v, table, kv_len, device_status=st)
    assert int(st.item()) == 0 and torch.isfinite(o["out"].float()).all()
    # against plain attention in float64 over the gathered cache
    kk, vv = (x[table[0].long()].view(-1, 64).double() for x in (k, v))
    z = (q[0].double().view(-1, 64) @ kk.T) * 0.125
    keep = torch.arange(num * 8, device=DEV)[None, :] <= num * 8 - n + torch.arange(
        n, device=DEV).repeat_interleave(hq)[:, None]
    w = torch.softmax(torch.where(keep, z, float("-inf")), -1)
    ref, absv = w @ vv, w @ vv.abs()
    # 7e5 terms of the sums and a maximum that may grow in each of their tiles,
    # and half a step of bf16 for the weights and for the result
    tol = absv * (2 * 7.2e5 * 1.4 * 2.0 ** -24 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    assert ((o["out"][0].double().view(-1, 64) - ref).abs() <= tol).all()
    for at in (5, 44321, num - 1):
        bad = table.clone()
        bad[0, at] = num
        st.zero_()
        o = sv.sv_kv_attend(q, k, v, bad, kv_len, device_status=st)
        assert int(st.item()) == sv.SV_DEV_BAD_INDEX and torch.isnan(o["out"]).all()


def test_attend_offsets_past_32_bits():
    """Pages more than 2^31 elements apart."""
    far = (1 << 31) // 2 + 4096
    kc = torch.zeros(2 * far + 16 * 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    k = kc.as_strided((3, 16, 1, 128), (far, 128, 128, 1))
    v = vc.as_strided((3, 16, 1, 128), (far, 128, 128, 1))
    g = torch.Generator(device=DEV).manual_seed(0)
    for t in (k, v):
        t.copy_(torch.randn(3, 16, 1, 128, generator=g, device=DEV))
    for n, hq in ((1, 4), (4, 16), (9, 8)):
        s = dict(q=torch.randn(1, n, hq, 128, generator=g, device=DEV).bfloat16(), kc=k, vc=v,
                 table=[[2, 0, 1]], kv_len=[48 - n], q_len=[n], parents=None, scale=128 ** -0.5,
                 page=16)
        out, lse, st = call_attend(s)
        assert st == 0
        check_attend(s, out, lse)
    slots = torch.tensor([[2 * 16 + 5]], device=DEV)
    x = torch.randn(1, 1, 1, 128, device=DEV).bfloat16()
    sv.sv_kv_append(x, x, slots, k, v)
    assert torch.equal(k[2, 5], x[0, 0]) and torch.equal(v[2, 5], x[0, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["chain", "line", "bush"])
def test_attend_the_largest_step(dtype, shape):
    """1024 new tokens: a chain, the same as a tree of one line (the longest
    walks up), and a bush."""
    s = scenario(1, 1024, 2, 1, 64, 16, [70], dtype, seed=41)
    if shape == "line":
        s["parents"] = [[j - 1 for j in range(1024)]]
    elif shape == "bush":
        s["parents"] = [[-1] + [j // 3 if j % 7 else j - 1 for j in range(1, 1024)]]
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


def test_attend_a_prompt_in_pieces():
    """Pieces of a prompt, each over the whole of what stands before it, equal
    to rounding what one token at a time gives."""
    s = scenario(2, 300, 8, 2, 64, 16, [0, 33], "bf16", seed=43)
    whole, lw, _ = call_attend(s)
    for n, at in ((128, 0), (128, 128), (44, 256), (1, 299)):
        t = dict(s, q=s["q"][:, at:at + n], q_len=[n, n], kv_len=[x + at for x in s["kv_len"]])
        out, lse, st = call_attend(t)
        assert st == 0
        check_attend(t, out, lse)
        assert ((lse - lw[:, at:at + n]).abs() <= 1e-5 * (1 + lse.abs())).all()


@pytest.mark.parametrize("side", [False, True])
def test_a_step_captured_and_replayed(side):
    """plan, append, attend and commit in one graph, state in place: five
    replays leave the bits of five steps without a graph; on a side stream too."""
    B, n, page, mp, num = 6, 6, 4, 30, 200
    par = i32([[-1, 0, 0, 1, 1, 2]] * B)

    def fresh():
        g = torch.Generator(device=DEV).manual_seed(5)
        kc, vc = make_cache(num, page, 2, 64, torch.bfloat16, "dense", 7)
        x = torch.randn(B, n, 12, 64, generator=g, device=DEV).bfloat16()
        return dict(kv_len=i32([3, 0, 9, 4, 1, 7]), pages=i32([1, 0, 3, 1, 1, 2]),
                    count=i32([num - 8]), written=i32([0] * B), free=i32(
                        list(range(8, num)) + [-1] * 8),
                    table=i32([r + [-1] * (mp - len(r)) for r in (
                        [0], [], [1, 2, 3], [4], [5], [6, 7])]),
                    acc=i32([2, 1, 0, 2, 1, 0]), new=i32([6, 6, 1, 6, 3, 0]),
                    nodes=i32([[0, 2, 5], [0, 1, -1], [0, -1, -1], [0, 1, 4], [0, 2, -1],
                               [0, -1, -1]]), x=x, kc=kc, vc=vc, st=status())

    def step(s, stream=None):
        o = sv.sv_kv_plan(s["kv_len"], s["table"], s["pages"], s["free"], s["count"], s["new"], n,
                          page, written=s["written"], accepted_len=s["acc"], stream=stream,
                          out=dict(kv_len=s["kv_len"], pages=s["pages"], free_count=s["count"],
                                   q_len=s["written"]), device_status=s["st"])
        sv.sv_kv_append(s["x"][:, :, 8:10], s["x"][:, :, 10:], o["slot_map"], s["kc"], s["vc"],
                        device_status=s["st"], stream=stream)
        a = sv.sv_kv_attend(s["x"][:, :, :8], s["kc"], s["vc"], s["table"], s["kv_len"],
                            q_len=s["written"], parents=par, device_status=s["st"], stream=stream)
        s["x"].copy_(torch.cat([a["out"], s["x"][:, :, :4]], 2))  # the next step's inputs
        sv.sv_kv_commit(s["kc"], s["vc"], s["table"], s["kv_len"], s["nodes"], s["acc"],
                        device_status=s["st"], stream=stream)

    want, got = fresh(), fresh()
    # tokens 0 .. accepted of a request that writes fewer are the last step's
    for s in (want, got):
        s["acc"].copy_(torch.minimum(s["acc"], (s["new"] - 1).clamp(min=0)))
    stream = torch.cuda.Stream()
    for _ in range(5):
        if side:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                step(want, stream)
            torch.cuda.current_stream().wait_stream(stream)
        else:
            step(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    state = {k: v.clone() for k, v in got.items()}
    with torch.cuda.graph(g):
        step(got)
    for k, v in state.items():
        got[k].copy_(v)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert int(want["st"].item()) == 0
    for k in want:
        bits = torch.int16 if want[k].dtype == torch.bfloat16 else want[k].dtype
        assert torch.equal(want[k].view(bits), got[k].view(bits)), k


@pytest.mark.parametrize("n,g", [(1, 4), (2, 4), (4, 4)])
def test_attend_fp32_sums_do_not_drift(n, g):
    """Blocks that add up 250 steps of keys: roundings to nearest, independent,
    give an error of about sqrt(250) 2^-24 of the output, with the products' 20
    2^-24 below 2e-6; sums that are cut off would give 250 * 2^-24 / 2 and more,
    7e-6 (the norm of the error against the norm of the output)."""
    B, L, hkv, d = 64, 8000, 4, 64
    gen = torch.Generator(device=DEV).manual_seed(3)
    k = torch.randn(B * L // 16, 16, hkv, d, generator=gen, device=DEV)
    v = torch.rand(k.shape, generator=gen, device=DEV)  # of one sign
    q = torch.randn(B, n, hkv * g, d, generator=gen, device=DEV)
    table = torch.arange(B * L // 16, device=DEV, dtype=torch.int32).view(B, -1)
    o = sv.sv_kv_attend(q, k, v, table, i32([L - n] * B))["out"]
    err = ref2 = 0.0
    for b in (0, 31, 63):
        kk, vv = (x.view(B, L, hkv, d)[b].double().transpose(0, 1) for x in (k, v))
        qq = q[b].double().view(n, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, n * g, d)
        z = qq @ kk.transpose(1, 2) * d ** -0.5
        keep = torch.arange(L, device=DEV)[None, :] <= L - n + torch.arange(
            n, device=DEV).repeat_interleave(g)[:, None]
        r = torch.softmax(torch.where(keep, z, float("-inf")), -1) @ vv
        r = r.view(hkv, n, g, d).permute(1, 0, 2, 3).reshape(n, hkv * g, d)
        err += float(((o[b].double() - r) ** 2).sum())
        ref2 += float((r ** 2).sum())
    assert (err / ref2) ** 0.5 < 2e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_repeats_bit_for_bit_whatever_its_scratch_holds(dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for n, hq, lens in ((1, 4, [9000, 30, 1]), (4, 16, [5000, 77, 3]), (8, 16, [5000, 77, 3]),
                        (20, 16, [2000, 9, 4000])):
        s = scenario(3, n, hq, 2, 128, 16, lens, dtype, seed=2)
        nb = sv.sv_kv_attend_scratch_size(3, n, hq, 2, 128, dt)
        first = call_attend(s)
        for fill in (0, 0x7F, 0xFF):
            scratch = torch.full((nb,), fill, dtype=torch.uint8, device=DEV)
            again = call_attend(s, scratch=scratch)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_attend_on_two_streams_at_once():
    a = scenario(2, 4, 16, 2, 128, 16, [9000, 5000], "bf16", seed=2)
    b = scenario(2, 4, 16, 2, 128, 16, [8000, 6000], "bf16", seed=3)
    want = [call_attend(x)[:2] for x in (a, b)]
    args = [(x["q"], x["kc"], x["vc"], i32(x["table"]), i32(x["kv_len"])) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for j in range(2):
            got[j].append(sv.sv_kv_attend(*args[j], stream=streams[j]))
    torch.cuda.synchronize()
    for j in range(2):
        for o in got[j]:
            assert torch.equal(o["out"], want[j][0]) and torch.equal(o["lse"], want[j][1])


def test_attend_captured_and_replayed_with_new_lengths():
    s = scenario(3, 4, 16, 2, 128, 16, [900, 400, 64], "bf16", seed=2)
    table, kv_len = i32(s["table"]), i32(s["kv_len"])
    outs = []
    graphs = []
    for _ in range(2):  # two graphs of the same call, replayed at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sv.sv_kv_attend(s["q"], s["kc"], s["vc"], table, kv_len))
        graphs.append(g)
    # the second set asks request 1 for pages it does not hold: NaN, as uncaptured
    for lens in ([900, 400, 64], [0, 800, 1], [5, 5, 5]):
        kv_len.copy_(i32(lens))
        want = sv.sv_kv_attend(s["q"], s["kc"], s["vc"], table, kv_len)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            for k, bits in (("out", torch.int16), ("lse", torch.int32)):
                assert torch.equal(o[k].view(bits), want[k].view(bits))


@pytest.mark.parametrize("n,d,lens", [(10, 128, [900, 300, 64]), (40, 64, [20, 2000, 64]),
                                      (20, 128, [5000])])
def test_attend_bounded_wait_runs_out_and_reports(n, d, lens):
    """The test hook leaves out one copy: the waits for it give up after 20 ms,
    the call returns, the first block's rows are NaN, the last request is
    whole, and so is the next call."""
    s = scenario(4, n, 8, 2, d, 16, lens, "bf16", seed=31)
    clean = call_attend(s)
    assert clean[2] == 0
    with sv.knobs(wait_ns=20_000_000, stall=1):
        out, lse, st = call_attend(s)
    assert st == sv.SV_DEV_TIMEOUT and sv.sv_device_status_check(st) == sv.SV_ERR_TIMEOUT
    assert torch.isnan(out[0, 0, 0]).all() and torch.isnan(lse[0, 0, 0])
    assert torch.equal(out[3], clean[0][3]) and torch.equal(lse[3], clean[1][3])
    again = call_attend(s)
    assert again[2] == 0 and torch.equal(again[0], clean[0]) and torch.equal(again[1], clean[1])


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def random_path(rng, n, a):
    return [0] + sorted(rng.sample(range(1, n), a))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,layers,n,heads,d,page,dtype", [
    (1, 1, 2, 1, 1, 1, "f32"), (4, 3, 32, 2, 64, 16, "bf16"), (7, 2, 40, 3, 20, 3, "bf16"),
    (2, 1, 1000, 1, 128, 64, "bf16"), (70, 4, 12, 1, 256, 5, "f32")])
def test_commit_matches_the_oracle(B, layers, n, heads, d, page, dtype, layout):
    rng = random.Random(B + n)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kv_len = [rng.randint(0, 3 * page) for _ in range(B)]
    cnt = [-(-(a + n) // page) for a in kv_len]
    ids = list(range(sum(cnt) + 2))
    rng.shuffle(ids)
    table, at = [], 0
    for c in cnt:
        table.append(ids[at:at + c] + [-1] * (max(cnt) - c))
        at += c
    caches = [make_cache(len(ids), page, heads, d, dt, layout, j) for j in range(layers)]
    kc = torch.stack([c[0] for c in caches])
    vc = torch.stack([c[1] for c in caches])
    if layout == "joint":  # keep the layout: layers of joint pages
        t = torch.stack([torch.stack([a, b], 1) for a, b in caches])
        kc, vc = t[:, :, 0], t[:, :, 1]
    elif layout == "heads_first":
        kc, vc = (torch.stack([c[j].transpose(1, 2).contiguous() for c in caches]).transpose(2, 3)
                  for j in range(2))
    alen = [rng.choice([-1, 0, rng.randint(0, n - 1), n - 1]) for _ in range(B)]
    width = max(max(alen) + 1, 1)
    nodes = [random_path(rng, n, max(a, 0)) + [-1] * (width - max(a, 0) - 1) for a in alen]
    want = [O.commit(host(c), table, kv_len, nodes, alen) for c in (kc, vc)]
    st = status()
    if layers == 1:
        sv.sv_kv_commit(kc[0], vc[0], i32(table), i32(kv_len), i32(nodes), i32(alen),
                        device_status=st)
    else:
        sv.sv_kv_commit(kc, vc, i32(table), i32(kv_len), i32(nodes), i32(alen), device_status=st)
    assert int(st.item()) == 0
    assert np.array_equal(host(kc), want[0]) and np.array_equal(host(vc), want[1])


@pytest.mark.parametrize("change,bit", [
    (dict(nodes=[0, 3, 2]), sv.SV_DEV_BAD_TREE), (dict(nodes=[0, 3, 3]), sv.SV_DEV_BAD_TREE),
    (dict(nodes=[1, 2, 3]), sv.SV_DEV_BAD_TREE), (dict(nodes=[0, -1, 3]), sv.SV_DEV_BAD_TREE),
    (dict(nodes=[0, 2, 60]), sv.SV_DEV_BAD_LEN), (dict(alen=3), sv.SV_DEV_BAD_LEN),
    (dict(kv_len=-1), sv.SV_DEV_BAD_LEN), (dict(page=99), sv.SV_DEV_BAD_INDEX)])
def test_commit_refuses_bad_paths_whole(change, bit):
    c = dict(nodes=[0, 2, 5], alen=2, kv_len=3, page=0)
    c.update(change)
    kc, vc = make_cache(6, 4, 1, 16, torch.bfloat16, "dense", 1)
    before = kc.clone(), vc.clone()
    st = status()
    sv.sv_kv_commit(kc, vc, i32([[5, 4, c["page"]], [1, 2, 3]]), i32([c["kv_len"], 0]),
                    i32([c["nodes"], [0, 2, -1]]), i32([c["alen"], 1]), device_status=st)
    assert int(st.item()) == bit
    want = [x.clone() for x in before]
    for x in want:
        x[1, 1] = x[1, 2]  # the sound request's move
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


# ---------------------------------------------------------------------------
# refusals that need device tensors
# ---------------------------------------------------------------------------
def test_binding_refuses_mismatched_tensors():
    s = scenario(2, 2, 4, 2, 64, 16, [10, 20], "bf16")
    t, l = i32(s["table"]), i32(s["kv_len"])

    def attend(**kw):
        a = dict(q=s["q"], kc=s["kc"], vc=s["vc"], t=t, l=l)
        a.update(kw)
        rest = {k: a.pop(k) for k in list(a) if k not in ("q", "kc", "vc", "t", "l")}
        return sv.sv_kv_attend(a["q"], a["kc"], a["vc"], a["t"], a["l"], **rest)
    for kw in (dict(q=s["q"].float()), dict(q=s["q"][..., :32]), dict(q=s["q"].transpose(2, 3)),
               dict(vc=s["vc"].float()), dict(vc=s["vc"][:-1]), dict(t=t[:1]), dict(l=l[:1]),
               dict(q_len=l[:1]), dict(parents=t[:, :1].contiguous()), dict(t=t[0]),
               dict(vc=s["vc"].transpose(1, 2).contiguous().transpose(1, 2)),
               dict(out=dict(out=torch.empty(1, device=DEV, dtype=torch.bfloat16)))):
        with pytest.raises((TypeError, ValueError)):
            attend(**kw)
    with pytest.raises(TypeError):
        attend(l=l.long())
    with pytest.raises(sv.SVError) as e:
        attend(scratch=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == sv.SV_ERR_WORKSPACE
    with pytest.raises(sv.SVError) as e:
        attend(q=s["q"][:, :, :3].contiguous())  # 3 query heads over 2 key heads
    assert e.value.status == sv.SV_ERR_INVALID_ARG
    for kw in (dict(scale=float("inf")), dict(out=dict(out=s["q"]))):  # out over q
        with pytest.raises(sv.SVError) as e:
            attend(**kw)
        assert e.value.status == sv.SV_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# a run of them together, with the verification calls
# ---------------------------------------------------------------------------
class Model:
    """A one-layer attention model with tied weights: enough for the cache to
    matter, small enough to recompute densely in float64."""

    def __init__(self, V, hq, hkv, d, seed):
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hkv, self.d, self.V = hq, hkv, d, V
        self.emb = torch.randn(V, (hq + 2 * hkv) * d, generator=g).bfloat16().to(DEV)
        self.head = (torch.randn(hq * d, V, generator=g) / (hq * d) ** 0.5).to(DEV)

    def qkv(self, tokens):
        x = self.emb[tokens.clamp(min=0)].view(*tokens.shape, self.hq + 2 * self.hkv, self.d)
        return x[:, :, :self.hq], x[:, :, self.hq:self.hq + self.hkv], x[:, :, self.hq + self.hkv:]

    def logits(self, o):
        return 3.0 * (o.float().flatten(2) @ self.head)

    def dense(self, seq):
        """Logits after the last token of a sequence, without a cache."""
        x = host(self.emb[torch.tensor(seq, device=DEV)]).reshape(len(seq), -1, self.d)
        g = self.hq // self.hkv
        o = []
        for h in range(self.hq):
            k, v = x[:, self.hq + h // g], x[:, self.hq + self.hkv + h // g]
            z = k @ x[-1, h] * self.d ** -0.5
            w = np.exp(z - z.max())
            o.append(w @ v / w.sum())
        o = host(torch.tensor(np.concatenate(o)).bfloat16())  # the layer's output type
        return 3.0 * o @ host(self.head)


@pytest.mark.parametrize("tree", [False, True])
def test_speculative_decoding_through_the_cache(tree):
    """Prompts, then steps of drafting, attending, greedy verification and
    commit until every request has 20 tokens: the tokens are those that greedy
    decoding without a cache gives, and all pages come back at the end."""
    V, page, B, mp, target = 37, 4, 5, 20, 20
    m = Model(V, 4, 2, 64, 0)
    rng = random.Random(4)
    prompts = [[rng.randrange(V) for _ in range(rng.randint(1, 9))] for _ in range(B)]
    seqs = [list(x) for x in prompts]
    want = []
    for x in prompts:
        y = list(x)
        for _ in range(target + 8):
            z = m.dense(y)
            y.append(int(np.argmax(z)))
        want.append(y)
    num = 60
    kc, vc = make_cache(num, page, 2, 64, torch.bfloat16, "heads_first", 0, fill=float("nan"))
    table = i32([[-1] * mp] * B)
    free, count = i32(list(range(num))[::-1]), i32([num])
    kv_len, pages = i32([0] * B), i32([0] * B)
    written, accepted = i32([0] * B), i32([0] * B)
    done = [False] * B
    st = status()

    def plan(new, mx, release=None):
        nonlocal kv_len, pages, count, written
        o = sv.sv_kv_plan(kv_len, table, pages, free, count, i32(new), mx, page, written=written,
                          accepted_len=accepted, release=release,
                          out=dict(kv_len=kv_len, pages=pages, free_count=count, q_len=written),
                          device_status=st)
        return o

    def forward(tokens, o, parents=None):
        q, k, v = m.qkv(tokens)
        sv.sv_kv_append(k, v, o["slot_map"], kc, vc, device_status=st)
        a = sv.sv_kv_attend(q, kc, vc, table, o["kv_len"], q_len=o["q_len"], parents=parents,
                            device_status=st)
        return m.logits(a["out"]).contiguous()

    # prompts: all but the last token of each, whose logits a step computes
    mx = max(map(len, prompts))
    o = plan([len(x) - 1 for x in prompts], mx)
    toks = torch.zeros(B, mx, dtype=torch.long, device=DEV)
    for b, x in enumerate(prompts):
        toks[b, :len(x)] = torch.tensor(x, device=DEV)
    forward(toks, o)
    accepted = torch.where(written > 0, written - 1, 0).to(torch.int32)
    while not all(done):
        n = 7 if tree else 4
        par = [-1, 0, 0, 1, 1, 2, 2]
        toks = torch.zeros(B, n, dtype=torch.long, device=DEV)
        for b in range(B):
            toks[b, 0] = seqs[b][-1]
            nxt = want[b][len(seqs[b]):]
            for j in range(1, n):
                depth = j if not tree else (1 if j < 3 else 2)
                right = rng.random() < 0.6 and (not tree or j in (2, 5, 6))
                toks[b, j] = nxt[depth - 1] if right else rng.randrange(V)
            if tree and int(toks[b, 1]) == int(toks[b, 2]):
                toks[b, 1] = (int(toks[b, 2]) + 1) % V
            if tree and int(toks[b, 5]) == int(toks[b, 6]):
                toks[b, 6] = (int(toks[b, 5]) + 1) % V
        rel = i32([int(x) for x in done])
        o = plan([0 if x else n for x in done], n, release=rel)
        lg = forward(toks, o, i32([par] * B) if tree else None)
        if tree:
            r = sv.sv_verify_tree_greedy(lg, toks.to(torch.int32).contiguous(), i32([par] * B), 2,
                                         device_status=st)
            sv.sv_kv_commit(kc, vc, table, o["kv_len"], r["accepted_nodes"], torch.where(
                o["q_len"] > 0, r["accepted_len"], -1).to(torch.int32), device_status=st)
        else:
            r = sv.sv_verify_chain_ragged(lg, None, toks[:, 1:].to(torch.int32).contiguous(), None,
                                          0.0, active=o["q_len"], device_status=st)
        accepted = r["accepted_len"]
        for b in range(B):
            if not done[b]:
                a = int(accepted[b])
                seqs[b] += r["out_tokens"][b, :a + 1].tolist()
                done[b] = len(seqs[b]) - len(prompts[b]) >= target
    o = plan([0] * B, 1, release=i32([1] * B))
    assert int(st.item()) == 0
    assert int(count.item()) == num and sorted(free.tolist()) == list(range(num))
    for b in range(B):
        k = min(len(seqs[b]), len(want[b]))
        assert seqs[b][:k] == want[b][:k]
