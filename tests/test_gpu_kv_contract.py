"""What the header promises of the paged cache calls, beside the agreement with
the oracle: precision of long contexts and of many rows, values that are not
finite, requests that a step leaves out, bad page ids, limits of sizes."""
import os
import subprocess
import sys

import pytest
import torch

from oracle import kv
from speculative_decoding_verification_94_b200 import sv
from tests.test_gpu_kv import (DEV, call_attend, check_attend, check_plan, i32, run_plan, scenario,
                               status)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def exact(s):
    """(out, lse) of a scenario in float64, and sum p |v|; zeros and -inf for
    tokens behind a request's own."""
    q, kc, vc, page = s["q"].double(), s["kc"], s["vc"], s["page"]
    B, n, hq, d = q.shape
    heads = kc.shape[2]
    g = hq // heads
    out, absv = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, n, hq), float("-inf"), dtype=torch.float64, device=q.device)
    for b in range(B):
        a, m = s["kv_len"][b], s["q_len"][b]
        if m == 0:
            continue
        keep = torch.ones(m, a + m, dtype=torch.bool)
        for i in range(m):
            keep[i, a:] = False
            j = i
            while j >= 0:
                keep[i, a + j] = True
                j = j - 1 if s["parents"] is None else s["parents"][b][j]
        keep = keep.to(q.device).repeat_interleave(g, 0)
        ids = torch.tensor(s["table"][b][:-(-(a + m) // page)], device=q.device)
        for h in range(heads):
            k = kc[ids, :, h].reshape(-1, d)[:a + m].double()
            v = vc[ids, :, h].reshape(-1, d)[:a + m].double()
            z = q[b, :m, h * g:(h + 1) * g].reshape(m * g, d) @ k.T * s["scale"]
            z = torch.where(keep, z, float("-inf"))
            w = torch.softmax(z, -1)
            out[b, :m, h * g:(h + 1) * g] = (w @ v).view(m, g, d)
            absv[b, :m, h * g:(h + 1) * g] = (w @ v.abs()).view(m, g, d)
            lse[b, :m, h * g:(h + 1) * g] = torch.logsumexp(z, -1).view(m, g)
    return out, lse, absv


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,g", [(4, 7), (8, 5), (16, 4), (16, 8), (32, 8)])
def test_attend_bf16_errs_by_its_outputs_rounding_alone(n, g, d, tree):
    """The weights enter the product as two bf16, to 2^-16 of each: with
    sum p |v| some ten times an output's size that is 1.5e-4 of the output,
    scores in fp32 add as much, and the output's own rounding 1.7e-3.  They add
    up as squares to 2 % more than the rounding of the exact output; 5 % are
    allowed.  (Weights of one bf16 would add another 1.3e-3: 27 % more.)"""
    s = scenario(2, n, 2 * g, 2, d, 16, [700, 2500], "bf16", tree=tree, seed=3 * n + d)
    out, lse, st = call_attend(s)
    assert st == 0
    ref = exact(s)[0]
    least = float((ref.bfloat16().double() - ref).norm())
    assert float((out.double() - ref).norm()) <= 1.05 * least


@pytest.mark.parametrize("n,hq,d", [(1, 1, 64), (1, 4, 128), (2, 8, 128), (5, 8, 64)])
def test_attend_of_the_shortest_segments_repeats(n, hq, d):
    """One to three keys a request, so that a block's warps end their first
    segment as soon as they can: the same bits in every call, and right ones."""
    s = scenario(600, n, hq, 1, d, 16, [0, 2, 1], "bf16", ragged=True, seed=n + d)
    want = call_attend(s)
    ref, lse, absv = exact(s)
    # three keys: 2^-16 of the weights, scores and powers to 300 half steps of
    # fp32 of a score's size (below 100), half a step of the output
    tol = absv * (2.0 ** -16 + 2 * 300 * 100 * 2.0 ** -24) + 2.0 ** -8 * ref.abs() + 1e-30
    assert want[2] == 0 and ((want[0].double() - ref).abs() <= tol).all()
    args = (s["q"], s["kc"], s["vc"], i32(s["table"]), i32(s["kv_len"]))
    for _ in range(200):
        o = sv.sv_kv_attend(*args, q_len=i32(s["q_len"]), scale=s["scale"])
        assert torch.equal(o["out"], want[0]) and torch.equal(o["lse"], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_commit_moves_nothing_of_a_request_that_the_step_left_out(dtype):
    """Request 0 ends and its pages go to request 1 in the same plan; the tree
    call still finds it an accepted path."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    table, free = i32([[0, 1, -1], [2, -1, -1]]), i32([-1, -1, -1])
    o = sv.sv_kv_plan(i32([6, 4]), table, i32([2, 1]), free, i32([0]), i32([0, 7]), 7, 4,
                      written=i32([0, 0]), accepted_len=i32([0, 0]), release=i32([1, 0]))
    assert table.tolist() == [[0, 1, -1], [2, 1, 0]] and o["q_len"].tolist() == [0, 7]
    g = torch.Generator(device=DEV).manual_seed(0)
    kc, vc = (torch.randn(2, 3, 4, 1, 8, generator=g, device=DEV).to(dt) for _ in range(2))
    want = kc.clone(), vc.clone()
    for w in want:  # request 1: position 5 (page 1) takes position 8 (page 0)
        w[:, 1, 1] = w[:, 0, 0]
    st = status()
    sv.sv_kv_commit(kc, vc, table, o["kv_len"], i32([[0, 2], [0, 4]]), i32([1, 1]),
                    q_len=o["q_len"], device_status=st)
    assert int(st.item()) == 0
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


@pytest.mark.parametrize("q,bit", [([3, 6, 0], 0), ([2, 6, 0], sv.SV_DEV_BAD_TREE),
                                   ([1, 6, 5], sv.SV_DEV_BAD_TREE),
                                   ([-1, 6, 0], sv.SV_DEV_BAD_LEN), (None, 0)])
def test_commit_moves_no_node_that_was_not_written(q, bit):
    g = torch.Generator(device=DEV).manual_seed(1)
    kc = torch.randn(8, 4, 2, 8, generator=g, device=DEV)
    vc = torch.randn(8, 4, 2, 8, generator=g, device=DEV)
    want = kc.clone(), vc.clone()
    for w in want:
        if q is None or q[0] == 3:
            w[0, 1] = w[0, 2]           # request 0: node 2 to position 1
        w[2, 2], w[2, 3] = w[2, 3].clone(), w[3, 2].clone()  # request 1: nodes 2, 5 behind 1 token
        if q is None or q[2] == 5:
            w[5, 1] = w[5, 3]           # request 2: node 3
    st = status()
    sv.sv_kv_commit(kc, vc, i32([[0, 1], [2, 3], [5, 6]]), i32([0, 1, 0]),
                    i32([[0, 2, -1], [0, 2, 5], [0, 3, -1]]), i32([1, 2, 1]),
                    q_len=None if q is None else i32(q), device_status=st)
    assert int(st.item()) == bit
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


@pytest.mark.parametrize("val", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("at", ["new", "committed"])
@pytest.mark.parametrize("n,hq,d,dtype", [
    (3, 4, 128, "f32"), (2, 8, 64, "f32"),                       # up to 8 rows
    (6, 12, 64, "f32"), (6, 12, 128, "f32"),                     # more
    (3, 4, 50, "f32"), (3, 4, 200, "f32"), (3, 4, 50, "bf16"),   # the general kernel
    (3, 4, 128, "bf16"), (20, 8, 64, "bf16"), (20, 16, 128, "bf16")])
def test_attend_values_that_are_not_finite_count_at_any_weight(n, hq, d, dtype, at, val):
    """A key whose weight underflows to zero, its value not finite: the element
    of the output is not finite for the rows that attend to it, and no other
    element or row changes."""
    s = scenario(2, n, hq, 2, d, 16, [5, 70], dtype, seed=23, q_scale=1.0)
    s["q"][..., 0] = 30.0
    for c in (s["kc"],):
        c[..., 0] = 4.0
    spots = []
    for b in range(2):
        pos = s["kv_len"][b] + 1 if at == "new" else s["kv_len"][b] - 1
        spots.append((s["table"][b][pos // 16], pos % 16))
        s["kc"][spots[-1]][:, 0] = -3000.0  # weight e^(-90000 / sqrt d) = 0
    first = 1 if at == "new" else 0         # the first row that attends to it
    clean, lse, st = call_attend(s)
    assert st == 0 and torch.isfinite(clean.float()).all()
    t = dict(s, vc=s["vc"].clone())
    for x in spots:
        t["vc"][x][:, 3] = val
    out, lse2, st = call_attend(t)
    assert st == 0 and torch.equal(lse, lse2)
    keep = [c for c in range(d) if c != 3]
    assert torch.equal(out[..., keep], clean[..., keep])
    assert torch.equal(out[:, :first], clean[:, :first])
    assert not torch.isfinite(out[:, first:, :, 3].float()).any()


@pytest.mark.parametrize("n,hq,d", [(2, 4, 64), (2, 4, 128), (6, 12, 64), (6, 12, 128), (3, 4, 50)])
def test_attend_fp32_queries_up_to_the_largest_number(n, hq, d):
    """q = +-FLT_MAX in one column, a scale that brings the scores back to a
    few: the same finite result whatever the number of rows."""
    s = scenario(2, n, hq, 2, d, 16, [5, 90], "f32", seed=29, q_scale=0.0)
    big = torch.finfo(torch.float32).max
    s["q"][..., 0] = big
    s["q"][:, :, ::2, 0] = -big
    s["kc"][..., 0] *= 0.2
    s["kc"][..., 0].clamp_(-0.9, 0.9)
    s["scale"] = 2.0 ** -126
    out, lse, st = call_attend(s)
    assert st == 0
    check_attend(s, out, lse)


FRESH_PLANS = """
import random, sys, torch
from oracle import kv as O
from tests.test_gpu_kv import check_plan, run_plan
from tests.test_kv_oracle import random_plan
for B in (1, 2026, 2027, 2048, 2049):
    args = random_plan(random.Random(B), B, 16, 12, 4, 900)
    got, st = run_plan(args, 16, 4)
    check_plan(got, O.plan(*args, 16, 4))
print("plans ok")
"""


def test_plan_of_2048_requests_is_the_first_of_its_process():
    """Batches whose shared memory passes 48 KB only with the kernel's own part,
    before any larger batch has raised the kernel's limit."""
    r = subprocess.run([sys.executable, "-c", FRESH_PLANS], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "plans ok" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("bad", [-1, 9, 1 << 30])
@pytest.mark.parametrize("release", [0, 1])
def test_plan_reports_a_bad_page_in_the_call_that_gives_it_back(bad, release):
    """Request 0 rolls back or ends; one of its pages is no page of the pool.
    Request 1 keeps its page and nobody takes one."""
    free = [7, 8] + [-9] * 7
    rel = None if not release else [1, 0]
    args = ([10, 4], [20, 0], [1, -1], rel, [0, 0], [[0, 1, bad, 3], [5, -7, -7, -7]], [2 + 2, 1],
            free, 2)
    got, st = run_plan(args, 8, 1)
    check_plan(got, kv.plan(*args, 8, 1))
    assert st == sv.SV_DEV_BAD_INDEX
    assert bad in got["free_pages"][:int(got["free_count"][0])]
    # the next plan, whose request takes it, says so again
    after = (got["kv_len"].tolist(), None, None, None, [0, 27], got["block_table"].tolist(),
             got["pages"].tolist(), got["free_pages"].tolist(), int(got["free_count"][0]))
    assert run_plan(after, 8, 27)[1] == sv.SV_DEV_BAD_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq,d", [(1, 4, 64), (20, 4, 64), (1, 5, 128), (5, 8, 128), (16, 8, 128)])
@pytest.mark.parametrize("keys", [31007, 130001, 719999])
def test_attend_long_contexts(keys, n, hq, d, dtype):
    """One request over nearly all blocks and a short one beside it.  Values of
    one sign that grow along the context, so that the output is of the size of
    sum p |v|: a lost or doubled part of a sequence (a 300th at least) moves lse
    by 3e-3, and parts in another order, or of another page, the output.

    bf16: rounding the exact output errs by 1.2e-3 to 1.7e-3 of its size, weights
    by 2^-16, and sums by a warp's run of at most 200 steps and the 300 parts
    joined, 500 2^-24 = 3e-5 in all: 5 % more than the rounding alone are allowed.
    fp32: the same 3e-5, and twice the score's error below.
    lse: 500 half steps, and (d + 4) + 20 half steps of a score's largest sum of
    |q k| (20 for products in two parts)."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    page, num = 16, -(-(keys + n) // 16)
    g = torch.Generator(device=DEV).manual_seed(keys + n)
    k = torch.randn(num + 4, page, 1, d, generator=g, device=DEV).to(dt)
    v = torch.rand(num + 4, page, 1, d, generator=g, device=DEV)
    order = torch.randperm(num, generator=g, device=DEV)
    where = torch.empty(num, device=DEV)
    where[order] = torch.arange(num, device=DEV) / num
    v[:num] += 2 * where[:, None, None, None]  # page j of the context: + 2 j / num
    v = v.to(dt)
    q = torch.randn(2, n, hq, d, generator=g, device=DEV).to(dt)
    table = torch.full((2, num), -1, dtype=torch.int32, device=DEV)
    table[0] = order.int()
    table[1, :3] = torch.tensor([num, num + 2, num + 1], dtype=torch.int32)
    lens = [keys, 17]
    st = status()
    o = sv.sv_kv_attend(q, k, v, table, i32(lens), device_status=st)
    assert int(st.item()) == 0
    eps = 2.0 ** -24
    for b in range(2):
        ids = table[b, :-(-(lens[b] + n) // page)].long()
        kk, vv = (x[ids].reshape(-1, d)[:lens[b] + n].double() for x in (k, v))
        qq = q[b].double().view(n * hq, d)
        z = qq @ kk.T * d ** -0.5
        size = float((qq.abs() @ kk.abs().T).amax()) * d ** -0.5
        see = lens[b] + torch.arange(n, device=DEV).repeat_interleave(hq)
        z[torch.arange(lens[b] + n, device=DEV)[None, :] > see[:, None]] = float("-inf")
        ref = torch.softmax(z, -1) @ vv
        err = float((o["out"][b].double().view(-1, d) - ref).norm() / ref.norm())
        score = (d + 24) * size * eps
        least = float((ref.to(dt).double() - ref).norm() / ref.norm())
        limit = 1.05 * least if dtype == "bf16" else least + 500 * eps + 2 * score
        assert limit < 2e-3 and err <= limit, (b, err, limit)
        off = (o["lse"][b].double().view(-1) - torch.logsumexp(z, -1)).abs().max()
        assert float(off) <= 500 * eps + score + 4 * eps * 20


@pytest.mark.parametrize("B,n", [(1, 3), (4, 1), (1, 1)])
def test_append_takes_any_stride_of_a_single_request_or_token(B, n):
    """k out of a rotary embedding (dense), v still a part of the projection:
    where they differ, there is one request or one token."""
    g = torch.Generator(device=DEV).manual_seed(2)
    fused = torch.randn(B, n, 6, 64, generator=g, device=DEV)
    v = fused[:, :, 4:]
    k = torch.randn(B * n * 2 * 64 * 9, generator=g, device=DEV)
    # k with v's strides where there is a choice to be taken, odd ones elsewhere
    k = k.as_strided((B, n, 2, 64), (v.stride(0) if B > 1 else 7, v.stride(1) if n > 1 else 11, 64, 1))
    kc, vc = torch.zeros(6, 4, 2, 64, device=DEV), torch.zeros(6, 4, 2, 64, device=DEV)
    slots = torch.arange(B * n, device=DEV).view(B, n) * 2 + 1
    sv.sv_kv_append(k, v, slots, kc, vc)
    for c, x in ((kc, k), (vc, v)):
        want = torch.zeros(24, 2, 64, device=DEV)
        want[slots.view(-1)] = x.reshape(-1, 2, 64)
        assert torch.equal(c.view(24, 2, 64), want)


@pytest.mark.parametrize("n,hq,dtype", [(1, 4, "bf16"), (6, 8, "bf16"), (1, 4, "f32"),
                                        (6, 8, "f32")])
def test_attend_strides_that_are_never_taken_change_nothing(n, hq, dtype):
    """One request, one page and one key head with odd strides of their own:
    the same kernel, so the same bits."""
    s = scenario(1, n, hq, 1, 64, 128, [100], dtype, seed=37, spare=0)
    want = call_attend(s)
    assert s["kc"].shape[0] == 1 and want[2] == 0
    odd = dict(s)
    odd["q"] = s["q"].as_strided(s["q"].shape, (12345,) + s["q"].stride()[1:])
    for name, page in (("kc", 3), ("vc", 5)):
        c = s[name]
        odd[name] = c.as_strided(c.shape, (page, c.stride(1), 2 * page + 1, 1))
    out, lse, st = call_attend(odd)
    assert st == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    st, old = status(), (s["kc"].clone(), s["vc"].clone())
    sv.sv_kv_commit(odd["kc"], odd["vc"], i32(s["table"]), i32([3]), i32([[0, 2, 5]]), i32([2]),
                    device_status=st)
    assert int(st.item()) == 0
    for c, was in zip((s["kc"], s["vc"]), old):
        was[0, 4], was[0, 5] = was[0, 5].clone(), was[0, 8].clone()
        assert torch.equal(c, was)


FIRST_IN_A_GRAPH = """
import torch
from speculative_decoding_verification_94_b200 import sv
from tests.test_gpu_kv import DEV, i32, scenario, status
sv.lib()
cases = []
for n, hq, dtype in ((1, 4, "bf16"), (8, 8, "bf16"), (20, 16, "bf16"), (2, 4, "f32"), (8, 8, "f32")):
    s = scenario(2, n, hq, 2, 64, 16, [30, 70], dtype, seed=n)
    cases.append((s, i32(s["table"]), i32(s["kv_len"])))
state = dict(kv=i32([3, 0]), table=i32([[0, -1], [-1, -1]]), pages=i32([1, 0]),
             free=i32([1, 2, 3, -1]), count=i32([3]), new=i32([2, 5]), nodes=i32([[0, 2], [0, 1]]),
             acc=i32([1, 1]), kc=torch.randn(4, 16, 1, 8, device=DEV), st=status())
state["vc"] = state["kc"].clone()
x = torch.randn(2, 5, 1, 8, device=DEV)
before = {k: v.clone() for k, v in state.items()}
def run():
    outs = [sv.sv_kv_attend(s["q"], s["kc"], s["vc"], t, l, device_status=state["st"])
            for s, t, l in cases]
    p = sv.sv_kv_plan(state["kv"], state["table"], state["pages"], state["free"], state["count"],
                      state["new"], 5, 16, device_status=state["st"])
    sv.sv_kv_append(x, x, p["slot_map"], state["kc"], state["vc"], device_status=state["st"])
    sv.sv_kv_commit(state["kc"], state["vc"], state["table"], p["kv_len"], state["nodes"],
                    state["acc"], q_len=p["q_len"], device_status=state["st"])
    return [o[k] for o in outs for k in ("out", "lse")] + list(p.values())
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
after = {k: v.clone() for k, v in state.items()}
for k, v in before.items():
    state[k].copy_(v)
want = run()
assert int(state["st"].item()) == int(after["st"].item())
for a, b in zip(got + list(after.values()), want + list(state.values())):
    assert torch.equal(a, b)
print("graph ok")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "graph ok" in r.stdout, r.stderr[-2000:]
