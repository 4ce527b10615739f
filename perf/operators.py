"""The paged key-value cache operators as they are measured: one pass of each
through its plain form (elementary torch operations) or through the library.

A speculative decoding step keeps the keys and values of every request in
pages of a shared pool.  Around the verification calls it
  - plans the step ("plan"): commits the accepted tokens, returns the pages of
    rejected drafts and finished requests, takes pages for the new tokens and
    maps every new token to its slot;
  - appends the new tokens' keys and values to their slots ("append");
  - attends from the new tokens (one, a drafted chain or a candidate tree) to
    the committed tokens and to their own ancestors ("attend");
  - after a tree was verified, moves the accepted path's keys and values to
    the front of the step's slots, in every layer ("commit").
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # attend ------------------------------------------------------------
        # one interactive request with a short context: latency
        dict(name="attend_decode_b1", op="attend", B=1, n=1, hq=28, hkv=4, d=128, page=16, lo=517,
             hi=517, dtype="bf16", tree=False, ragged=False, len_seed=1),
        # the chain verification batch (B = 32, k = 3): root and three drafts
        dict(name="attend_chain_b32", op="attend", B=32, n=4, hq=28, hkv=4, d=128, page=16,
             lo=700, hi=9000, dtype="bf16", tree=False, ragged=True, len_seed=2),
        # plain decoding of 16 x 16 rollouts, where speculation does not pay
        dict(name="attend_decode_b256", op="attend", B=256, n=1, hq=32, hkv=8, d=128, page=64,
             lo=100, hi=4000, dtype="bf16", tree=False, ragged=False, len_seed=3),
        # candidate trees of 32 nodes (B = 8)
        dict(name="attend_tree_b8", op="attend", B=8, n=32, hq=32, hkv=4, d=128, page=32, lo=2000,
             hi=8000, dtype="bf16", tree=True, ragged=False, len_seed=4),
        # the rollout tail: one request left, a long context, k = 7 drafts
        dict(name="attend_long_b1", op="attend", B=1, n=8, hq=40, hkv=8, d=128, page=16,
             lo=130001, hi=130001, dtype="bf16", tree=False, ragged=False, len_seed=5),
        # a small fp32 model, as parity runs use
        dict(name="attend_chain_f32", op="attend", B=4, n=4, hq=8, hkv=2, d=64, page=16, lo=300,
             hi=2500, dtype="f32", tree=False, ragged=True, len_seed=6),
        # plan --------------------------------------------------------------
        # between two verification steps of B = 32, k = 3
        dict(name="plan_verify_b32", op="plan", B=32, max_new=4, page=16, max_pages=640, lo=700,
             hi=9000, release=0.03, mode="verify", len_seed=7),
        # admitting 64 prompts of up to 2048 tokens beside 192 running requests
        dict(name="plan_prefill_b256", op="plan", B=256, max_new=2048, page=16, max_pages=1024,
             lo=0, hi=9000, release=0.1, mode="prefill", len_seed=8),
        # append ------------------------------------------------------------
        # the new tokens of one verification step
        dict(name="append_verify_b32", op="append", B=32, n=4, hkv=4, d=128, page=16,
             dtype="bf16", ragged=True, len_seed=9),
        # a prefill batch out of a fused projection's output
        dict(name="append_prefill_b32", op="append", B=32, n=2048, hkv=8, d=128, page=16,
             dtype="bf16", ragged=True, len_seed=10),
        # commit ------------------------------------------------------------
        # the accepted paths of B = 8 trees (n = 32, depth 5), 28 layers
        dict(name="commit_tree_b8", op="commit", B=8, n=32, depth=5, layers=28, hkv=4, d=128,
             page=32, lo=200, hi=1000, dtype="bf16", len_seed=11),
        # the same for 16 x 16 rollouts
        dict(name="commit_tree_b256", op="commit", B=256, n=32, depth=5, layers=28, hkv=4, d=128,
             page=16, lo=20, hi=120, dtype="bf16", len_seed=12),
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "plan", "append", "commit"])
    seed = rng.randint(1, 1 << 30)
    if op == "attend":
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 4, 5, 7, 8])
        d = rng.choice([64, 128])
        tree = rng.random() < 0.3
        n = _log(rng, 4, 64) if tree else _log(rng, 1, 16)
        hi = _log(rng, 16, 130000)
        budget = (1 << 30) // (2 * hkv * d * (4 if dtype == "f32" else 2))  # 1 GiB of cache
        B = _log(rng, 1, max(1, min(256, budget // hi)))
        return dict(op=op, B=B, n=n, hq=hkv * g, hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]),
                    lo=_log(rng, 1, hi), hi=hi, dtype=dtype, tree=tree,
                    ragged=rng.random() < 0.5, len_seed=seed)
    if op == "plan":
        page = rng.choice([16, 32, 64, 128])
        hi = _log(rng, 64, 16000)
        mode = rng.choice(["verify", "prefill"])
        max_new = _log(rng, 1, 32) if mode == "verify" else _log(rng, 33, 2048)
        return dict(op=op, B=_log(rng, 1, 256), max_new=max_new, page=page,
                    max_pages=-(-(hi + max_new + 64) // page), lo=0, hi=hi,
                    release=rng.uniform(0.0, 0.3), mode=mode, len_seed=seed)
    if op == "append":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, n=_log(rng, 1, max(1, 65536 // B)), hkv=rng.choice([1, 2, 4, 8]),
                    d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "f32"]), ragged=rng.random() < 0.5, len_seed=seed)
    n = _log(rng, 8, 64)
    return dict(op=op, B=_log(rng, 1, 128), n=n, depth=rng.randint(1, 6), layers=_log(rng, 1, 28),
                hkv=rng.choice([1, 2, 4]), d=rng.choice([64, 128]), page=rng.choice([16, 32]),
                lo=1, hi=_log(rng, 2, 200), dtype=rng.choice(["bf16", "f32"]), len_seed=seed)


def _esize(case):
    return 4 if case["dtype"] == "f32" else 2


def _lens(case):
    """Committed tokens and new tokens of each request."""
    r = random.Random(case["len_seed"])
    B, n = case["B"], case["n"]
    kv = [r.randint(case.get("lo", 0), case.get("hi", 0)) for _ in range(B)]
    if case.get("ragged"):
        # requests drafted fewer tokens, one of eight is idle
        new = [0 if r.random() < 0.125 else r.randint(max(1, n // 2), n) for _ in range(B)]
        new[0] = n
    else:
        new = [n] * B
    return kv, new


def _tree(case):
    """BFS-ordered candidate trees: parents[b][j] < j."""
    r = random.Random(case["len_seed"] + 77)
    B, n = case["B"], case["n"]
    out = []
    for _ in range(B):
        par, depth, kids = [-1], [0], [0]
        for j in range(1, n):
            # the first node that still has room, or a random later one
            cand = [i for i in range(j) if depth[i] < 5 and kids[i] < 8] or [j - 1]
            lo = par[-1] if par[-1] >= 0 else 0
            cand = [i for i in cand if i >= lo] or [j - 1]
            p = cand[min(int(r.random() * r.random() * len(cand)), len(cand) - 1)]
            par.append(p)
            depth.append(depth[p] + 1)
            kids.append(0)
            kids[p] += 1
        out.append(par)
    return out


def _paths(case):
    """Accepted paths of the trees: nodes root..best, ascending.  Every node
    is its own place on the path or lies past its end, as in wide trees, so
    that a second pass finds its sources unchanged."""
    r = random.Random(case["len_seed"] + 78)
    n, depth = case["n"], min(case["depth"], case["n"] // 2 - 1)
    out = []
    for _ in range(case["B"]):
        a = r.randint(0, depth)
        picks = sorted(r.sample(range(a + 1, n), a)) if a else []
        if picks and r.random() < 0.5:
            picks[0] = 1  # the first child of the root stays where it is
        out.append([0] + picks)
    return out


def _plan_host(case):
    """Host lists of a planning step: the state before it and its inputs."""
    r = random.Random(case["len_seed"])
    B, page, mp, mx = case["B"], case["page"], case["max_pages"], case["max_new"]
    cap = mp * page
    kv, written, accepted, new, release = [], [], [], [], []
    for b in range(B):
        fresh = case["mode"] == "prefill" and b % 4 == 0
        w = 0 if fresh else r.randint(1, min(mx, 32))
        length = 0 if fresh else min(r.randint(case["lo"], case["hi"]), cap - w)
        rel = 0 if fresh else int(r.random() < case["release"])
        acc = r.randint(0, w - 1) if w else 0
        nxt = 0 if rel else (r.randint(1, mx) if fresh or case["mode"] == "verify" else 1)
        nxt = min(nxt, cap - (length + acc + 1))
        kv.append(length)
        written.append(w)
        accepted.append(acc)
        new.append(max(nxt, 0))
        release.append(rel)
    pages = [-(-(kv[b] + written[b]) // page) for b in range(B)]
    grow = sum(max(0, -(-(kv[b] + accepted[b] + 1 + new[b]) // page) - pages[b]) for b in range(B))
    return kv, written, accepted, new, release, pages, grow + 64


# --------------------------------------------------------------------------
# what a pass has to read, write and compute
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        kv, written, accepted, new, release, pages, slack = _plan_host(case)
        B, page = case["B"], case["page"]
        moved = 0
        touched = 0  # table entries that the new tokens' slots come from
        for b in range(B):
            base = 0 if release[b] else kv[b] + (accepted[b] + 1 if written[b] else 0)
            need = -(-(base + new[b]) // page)
            moved += abs(need - pages[b])
            touched += need - base // page if new[b] else 0
        return {"bytes": 4 * B * 9 + 8 * moved + 4 * touched + 12 * B * case["max_new"],
                "flops": 0}
    es = _esize(case)
    if op == "append":
        _, new = _lens(case)
        t = sum(new)
        return {"bytes": 4 * t * case["hkv"] * case["d"] * es + 8 * case["B"] * case["n"],
                "flops": 0}
    if op == "commit":
        moves = sum(sum(1 for i, j in enumerate(p) if i != j) for p in _paths(case))
        row = case["hkv"] * case["d"] * es
        return {"bytes": 4 * moves * row * case["layers"] + 4 * case["B"] * (case["depth"] + 3),
                "flops": 0}
    kv, new = _lens(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    keys = sum(a + c for a, c in zip(kv, new) if c)
    pairs = sum(a * c + c * (c + 1) // 2 for a, c in zip(kv, new))
    rows = case["B"] * case["n"] * hq
    tables = sum(-(-(a + c) // page) for a, c in zip(kv, new) if c)
    return {"bytes": 2 * keys * hkv * d * es + (sum(new) * hq + rows) * d * es + 4 * rows +
                     4 * tables,
            "flops": 4 * pairs * hq * d}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _table(counts, max_pages, g, spare=5):
    """Block table of requests that hold counts[b] pages, in the scattered
    order that a used pool has; -1 past them."""
    total = sum(counts)
    ids = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    c = torch.tensor(counts, device=DEV)
    col = torch.arange(max_pages, device=DEV)[None, :]
    start = (torch.cumsum(c, 0) - c)[:, None]
    idx = (start + col).clamp(max=total + spare - 1)
    return torch.where(col < c[:, None], ids[idx], -1).contiguous(), ids, total


def _cache(shape, dtype, g, offset):
    """Keys carry per-channel offsets, as projections with a bias give them."""
    c = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    if offset:
        c += torch.randn(shape[-2:], generator=g, device=DEV, dtype=dtype)
    return c


def prepare(case, seed):
    g = _gen(seed)
    op, B, page = case["op"], case["B"], case["page"]
    st = dict(case=case)
    if op == "plan":
        kv, written, accepted, new, release, pages, slack = _plan_host(case)
        table, ids, held = _table(pages, case["max_pages"], g, slack)
        num = held + slack
        free = torch.full((num,), -1, dtype=torch.int32, device=DEV)
        free[:slack] = ids[held:]
        st.update(kv_len=_i32(kv), written=_i32(written), accepted_len=_i32(accepted),
                  new_len=_i32(new), release=_i32(release), pages=_i32(pages), block_table=table,
                  free_pages=free, free_count=_i32([slack]))
    else:
        dt = DTYPES[case["dtype"]]
        hkv, d, n = case["hkv"], case["d"], case["n"]
        kv, new = _lens(case)
        max_pages = -(-(max(kv) + n) // page)
        if op == "attend":
            counts = [-(-(a + c) // page) for a, c in zip(kv, new)]
            table, _, total = _table(counts, max_pages, g)
            q = 2.5 * torch.randn(B, n, case["hq"], d, generator=g, device=DEV)
            st.update(q=q.to(dt), k_cache=_cache((total + 5, page, hkv, d), dt, g, True),
                      v_cache=_cache((total + 5, page, hkv, d), dt, g, False), block_table=table,
                      kv_len=_i32(kv), q_len=_i32(new), kv_host=kv, new_host=new,
                      parents=_i32(_tree(case)) if case["tree"] else None,
                      parents_host=_tree(case) if case["tree"] else None,
                      scale=1.0 / math.sqrt(d))
        elif op == "append":
            # each request's new tokens follow a context of its own
            r = random.Random(case["len_seed"] + 5)
            kv = [r.randint(0, 3 * page) for _ in range(B)]
            counts = [-(-(a + c) // page) for a, c in zip(kv, new)]
            table, _, total = _table(counts, max(max(counts), 1), g)
            pos = torch.arange(n, device=DEV)[None, :] + _i32(kv)[:, None]
            pid = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1)).long()
            valid = torch.arange(n, device=DEV)[None, :] < _i32(new)[:, None]
            qkv = torch.randn(B, n, 4 * hkv, d, generator=g, device=DEV, dtype=dt)
            shape = (total + 5, page, hkv, d)
            st.update(k=qkv[:, :, 2 * hkv:3 * hkv], v=qkv[:, :, 3 * hkv:],
                      slot_map=torch.where(valid, pid * page + pos % page, -1).contiguous(),
                      k_cache=torch.zeros(shape, device=DEV, dtype=dt),
                      v_cache=torch.zeros(shape, device=DEV, dtype=dt))
        else:
            counts = [-(-(a + n) // page) for a in kv]
            table, _, total = _table(counts, max_pages, g)
            paths = _paths(case)
            width = max(case["depth"] + 1, max(len(p) for p in paths))
            shape = (case["layers"], total + 5, page, hkv, d)
            st.update(k_cache=_cache(shape, dt, g, False), v_cache=_cache(shape, dt, g, False),
                      block_table=table, kv_len=_i32(kv),
                      accepted_nodes=_i32([p + [-1] * (width - len(p)) for p in paths]),
                      accepted_len=_i32([len(p) - 1 for p in paths]), paths=paths, kv_host=kv)
    if own:
        from speculative_decoding_verification_94_b200 import sv
        st["sv"] = sv
        if op == "plan":
            st["out"] = dict(kv_len=torch.empty_like(st["kv_len"]),
                             pages=torch.empty_like(st["pages"]),
                             free_count=torch.empty_like(st["free_count"]),
                             q_len=torch.empty_like(st["new_len"]),
                             slot_map=torch.empty(B, case["max_new"], dtype=torch.int64,
                                                  device=DEV),
                             positions=torch.empty(B, case["max_new"], dtype=torch.int32,
                                                   device=DEV))
        elif op == "attend":
            st["out"] = dict(out=torch.empty_like(st["q"]),
                             lse=torch.empty(st["q"].shape[:3], dtype=torch.float32, device=DEV))
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_plan(s):
    o = s["sv"].sv_kv_plan(s["kv_len"], s["block_table"], s["pages"], s["free_pages"],
                           s["free_count"], s["new_len"], s["case"]["max_new"], s["case"]["page"],
                           written=s["written"], accepted_len=s["accepted_len"],
                           release=s["release"], out=s["out"])
    return (o["kv_len"], o["pages"], o["free_count"], o["q_len"], o["slot_map"], o["positions"],
            s["block_table"], s["free_pages"])


def _own_append(s):
    s["sv"].sv_kv_append(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"])
    return s["k_cache"], s["v_cache"]


def _own_attend(s):
    o = s["sv"].sv_kv_attend(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"],
                             q_len=s["q_len"], parents=s["parents"], scale=s["scale"],
                             out=s["out"])
    return o["out"], o["lse"]


def _own_commit(s):
    s["sv"].sv_kv_commit(s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"],
                         s["accepted_nodes"], s["accepted_len"])
    return s["k_cache"], s["v_cache"]


_OWN = dict(plan=_own_plan, append=_own_append, attend=_own_attend, commit=_own_commit)


def _plain_plan(s):
    page, mx = s["case"]["page"], s["case"]["max_new"]
    table, held, free = s["block_table"], s["pages"], s["free_pages"]
    num, mp = free.numel(), table.shape[1]
    commit = torch.where(s["written"] > 0, torch.minimum(s["accepted_len"] + 1, s["written"]), 0)
    base = torch.where(s["release"] != 0, 0, s["kv_len"] + commit)
    need = (base + s["new_len"] + page - 1) // page
    grow = (need - held).clamp(min=0)
    shrink = (held - need).clamp(min=0)
    top = s["free_count"] + shrink.sum()
    give = torch.cumsum(shrink, 0) - shrink
    take = torch.cumsum(grow, 0)
    granted = (grow == 0) | (take <= top)
    col = torch.arange(mp, device=table.device)[None, :]
    # surplus pages go onto the stack, in request order
    push = (col >= need[:, None]) & (col < held[:, None])
    to = torch.where(push, s["free_count"] + give[:, None] + col - need[:, None], num)
    stack = torch.cat([free, free[:1]])
    stack[to] = torch.where(push, table, stack[num])
    # and the new ones come off it
    pop = (col >= held[:, None]) & (col < need[:, None]) & granted[:, None]
    at = (top - 1 - (take - grow)[:, None] - (col - held[:, None])).clamp(0, num)
    table.copy_(torch.where(pop, stack[at], table))
    free.copy_(stack[:num])
    q_len = torch.where(granted, s["new_len"], 0)
    i = torch.arange(mx, device=table.device)[None, :]
    pos = base[:, None] + i
    pid = table.gather(1, (pos // page).clamp(max=mp - 1)).long()
    valid = i < q_len[:, None]
    slots = torch.where(valid, pid * page + pos % page, -1)
    left = top - torch.where(granted, take, 0).amax()
    return (base.to(torch.int32), torch.where(granted, need, held).to(torch.int32),
            left.to(torch.int32), q_len, slots, torch.where(valid, pos, -1).to(torch.int32),
            table, free)


def _plain_append(s):
    kc, vc, hd = s["k_cache"], s["v_cache"], s["k_cache"].shape[2:]
    slots = s["slot_map"].reshape(-1)
    keep = slots >= 0
    slots = slots[keep]
    kc.view(-1, *hd)[slots] = s["k"].reshape(-1, *hd)[keep]
    vc.view(-1, *hd)[slots] = s["v"].reshape(-1, *hd)[keep]
    return kc, vc


def _plain_attend(s):
    c = s["case"]
    q, kc, vc, page = s["q"], s["k_cache"], s["v_cache"], c["page"]
    B, n, hq, d = q.shape
    hkv = c["hkv"]
    g = hq // hkv
    out = torch.zeros_like(q)
    lse = torch.full((B, n, hq), float("-inf"), dtype=torch.float32, device=q.device)
    own_row = torch.arange(n, device=q.device)
    if s["parents"] is None:
        seen = (own_row[:, None] >= own_row[None, :]).expand(B, n, n)
    else:
        seen = torch.zeros(B, n, n, dtype=torch.bool, device=q.device)
        at = own_row.expand(B, n).clone()
        for _ in range(n):
            seen |= (at[:, :, None] == own_row)
            at = torch.where(at >= 0, s["parents"].long().gather(1, at.clamp(min=0)), -1)
    for b in range(B):
        a, m = s["kv_host"][b], s["new_host"][b]
        if m == 0:
            continue
        ids = s["block_table"][b, :-(-(a + m) // page)].long()
        k = kc[ids].reshape(-1, hkv, d)[:a + m].float().transpose(0, 1)
        v = vc[ids].reshape(-1, hkv, d)[:a + m].float().transpose(0, 1)
        qb = q[b, :m].float().reshape(m, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, m * g, d)
        z = (qb @ k.transpose(1, 2)) * s["scale"]
        hide = ~seen[b, :m, :m].repeat_interleave(g, 0)
        z[:, :, a:].masked_fill_(hide, float("-inf"))
        top = z.amax(-1, keepdim=True)
        p = torch.exp(z - top)
        tot = p.sum(-1, keepdim=True)
        o = (p @ v) / tot
        out[b, :m] = o.reshape(hkv, m, g, d).permute(1, 0, 2, 3).reshape(m, hq, d).to(q.dtype)
        w = (top + torch.log(tot)).reshape(hkv, m, g).permute(1, 0, 2)
        lse[b, :m] = w.reshape(m, hq)
    return out, lse


def _plain_commit(s):
    kc, vc, table = s["k_cache"], s["v_cache"], s["block_table"]
    page, hd = s["case"]["page"], s["k_cache"].shape[3:]
    nodes, alen = s["accepted_nodes"], s["accepted_len"]
    i = torch.arange(nodes.shape[1], device=table.device)[None, :]
    keep = (i <= alen[:, None]) & (nodes != i)
    src = s["kv_len"][:, None] + nodes.clamp(min=0)
    dst = (s["kv_len"][:, None] + i).clamp(max=table.shape[1] * page - 1)

    def slot(pos):
        return table.gather(1, (pos // page).long()).long() * page + pos % page
    src, dst = slot(src)[keep], slot(dst)[keep]
    for c in (kc, vc):
        flat = c.view(c.shape[0], -1, *hd)
        flat[:, dst] = flat[:, src]
    return kc, vc


_PLAIN = dict(plan=_plain_plan, append=_plain_append, attend=_plain_attend, commit=_plain_commit)


# --------------------------------------------------------------------------
# the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _EXACT[case["op"]](s, case)


def _exact_plan(s, case):
    page, mx = case["page"], case["max_new"]
    kv, written, acc, new, rel, pages, _ = _plan_host(case)
    table = s["block_table"].tolist()
    free = s["free_pages"].tolist()
    count = int(s["free_count"].item())
    B = case["B"]
    base, need = [], []
    for b in range(B):
        length = kv[b] + (min(acc[b] + 1, written[b]) if written[b] > 0 else 0)
        base.append(0 if rel[b] else length)
        need.append((base[b] + new[b] + page - 1) // page)
    for b in range(B):
        for j in range(need[b], pages[b]):
            free[count] = table[b][j]
            count += 1
    out_pages, q_len, starved = list(pages), list(new), False
    for b in range(B):
        grow = need[b] - pages[b]
        if grow > 0:
            starved = starved or grow > count
            if starved:
                q_len[b] = 0
                continue
            for j in range(pages[b], need[b]):
                count -= 1
                table[b][j] = free[count]
        out_pages[b] = need[b]
    slots = [[-1] * mx for _ in range(B)]
    poss = [[-1] * mx for _ in range(B)]
    for b in range(B):
        for i in range(q_len[b]):
            p = base[b] + i
            poss[b][i] = p
            slots[b][i] = table[b][p // page] * page + p % page
    return (_i32(base), _i32(out_pages), _i32([count]), _i32(q_len),
            torch.tensor(slots, dtype=torch.int64, device=DEV), _i32(poss), _i32(table),
            _i32(free))


def _exact_append(s, case):
    page = case["page"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    slots = s["slot_map"].cpu()
    for b in range(case["B"]):
        m = int((slots[b] >= 0).sum())
        where = slots[b, :m].to(DEV)
        kc[where // page, where % page] = s["k"][b, :m].double()
        vc[where // page, where % page] = s["v"][b, :m].double()
    return kc, vc


def _exact_attend(s, case):
    page, hkv, d, hq = case["page"], case["hkv"], case["d"], case["hq"]
    B, n = case["B"], case["n"]
    g = hq // hkv
    out = torch.zeros(B, n, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, hq), float("-inf"), dtype=torch.float64, device=DEV)
    table = s["block_table"].cpu()
    for b in range(B):
        a, m = s["kv_host"][b], s["new_host"][b]
        if m == 0:
            continue
        allow = torch.zeros(m, a + m, dtype=torch.bool)
        allow[:, :a] = True
        for i in range(m):
            j = i
            while j >= 0:
                allow[i, a + j] = True
                j = j - 1 if s["parents_host"] is None else s["parents_host"][b][j]
        allow = allow.to(DEV)
        ids = table[b, :-(-(a + m) // page)].long().to(DEV)
        for h in range(hkv):
            k = s["k_cache"][ids, :, h].reshape(-1, d)[:a + m].double()
            v = s["v_cache"][ids, :, h].reshape(-1, d)[:a + m].double()
            qh = s["q"][b, :m, h * g:(h + 1) * g].double().reshape(m * g, d)
            z = torch.matmul(qh, k.T) / math.sqrt(d)
            z = torch.where(allow.repeat_interleave(g, 0), z, float("-inf"))
            w = torch.logsumexp(z, -1)
            out[b, :m, h * g:(h + 1) * g] = (torch.exp(z - w[:, None]) @ v).reshape(m, g, d)
            lse[b, :m, h * g:(h + 1) * g] = w.reshape(m, g)
    return out, lse


def _exact_commit(s, case):
    page = case["page"]
    kc, vc = s["k_cache"], s["v_cache"]
    if kc.numel() > 1 << 30:
        return None  # the copies in 64 bits would not fit beside the passes
    table = s["block_table"].cpu()
    src, dst = [], []
    for b, path in enumerate(s["paths"]):
        for i, j in enumerate(path):
            for at, where in ((s["kv_host"][b] + j, src), (s["kv_host"][b] + i, dst)):
                where.append((int(table[b, at // page]), at % page))
    src, dst = torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV)
    out = []
    for c in (kc, vc):
        moved = c[:, src[:, 0], src[:, 1]].double()
        c = c.double()
        c[:, dst[:, 0], dst[:, 1]] = moved
        out.append(c)
    return tuple(out)


_EXACT = dict(plan=_exact_plan, append=_exact_append, attend=_exact_attend, commit=_exact_commit)
