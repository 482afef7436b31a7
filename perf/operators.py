"""Measured cases of the attention layers' operators: the paged key/value cache
(kv_reserve, kv_append, kv_commit) and the attention of a round's new tokens
over it (attn_verify).

A round of a hybrid stack takes the same drafted tokens through its recurrent
layers and its attention layers.  For the latter it reserves cache pages for
the new tokens (kv_reserve), writes each layer's keys and values into them
(kv_append), attends from the new tokens to everything cached and to
themselves, as a chain or along a draft tree (attn_verify), and, once the
accepted lengths are known, keeps the accepted path and gives back the pages
that it no longer needs (kv_commit).

Cache layouts: keys [L,P,Hkv,page,D]; values [L,P,Hkv,page/8,D,8], eight
tokens of a channel side by side.  Slot s is row s % page of page s / page.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's next token: a single sequence, one row per head
        dict(name="attend_one_token", op="attend", B=1, new_lo=1, new_hi=1, ctx_lo=777, ctx_hi=777,
             mix=1, Hq=32, Hkv=4, D=128, page=16, dtype="bf16", tree=False, pad=0),
        # a serving batch one token at a time, contexts from short to long
        dict(name="attend_tokens_long", op="attend", B=24, new_lo=1, new_hi=1, ctx_lo=500,
             ctx_hi=32000, mix=2, Hq=32, Hkv=4, D=128, page=64, dtype="bf16", tree=False, pad=0),
        # a verify round of 8 drafts over the 32 sequences of the stack workload
        dict(name="attend_drafts", op="attend", B=32, new_lo=8, new_hi=8, ctx_lo=400, ctx_hi=9000,
             mix=3, Hq=32, Hkv=4, D=128, page=64, dtype="bf16", tree=False, pad=0),
        # a verify round over 64-node draft trees, wide heads shared eight to one
        dict(name="attend_trees", op="attend", B=64, new_lo=64, new_hi=64, ctx_lo=300, ctx_hi=4000,
             mix=4, Hq=16, Hkv=2, D=256, page=32, dtype="bf16", tree=True, pad=0),
        # prompts of different lengths packed together, some behind a cached prefix
        dict(name="attend_prompts", op="attend", B=3, new_lo=1700, new_hi=4096, ctx_lo=150,
             ctx_hi=2500, mix=5, Hq=32, Hkv=4, D=128, page=64, dtype="bf16", tree=False, pad=13),
        # the 32-bit form, odd sizes, three query heads to one
        dict(name="attend_f32_ragged", op="attend", B=7, new_lo=3, new_hi=29, ctx_lo=0, ctx_hi=2500,
             mix=6, Hq=12, Hkv=4, D=64, page=16, dtype="f32", tree=False, pad=3),
        # pages for a verify round
        dict(name="reserve_drafts", op="reserve", B=32, new_lo=8, new_hi=8, ctx_lo=400, ctx_hi=9000,
             mix=7, page=64, short=False),
        # pages for a large mixed batch of prompts and single tokens
        dict(name="reserve_prompts", op="reserve", B=256, new_lo=1, new_hi=2048, ctx_lo=1,
             ctx_hi=16000, mix=8, page=16, short=False),
        # keys and values of a verify round
        dict(name="append_drafts", op="append", B=32, new_lo=8, new_hi=8, ctx_lo=40, ctx_hi=900,
             mix=9, L=1, Hkv=4, D=128, page=64, dtype="bf16"),
        # keys and values of a prompt batch
        dict(name="append_prompts", op="append", B=5, new_lo=1500, new_hi=6000, ctx_lo=1,
             ctx_hi=900, mix=10, L=1, Hkv=4, D=128, page=64, dtype="bf16"),
        # the end of a chain round: lengths and pages only
        dict(name="commit_drafts", op="commit", B=32, new_lo=8, new_hi=8, ctx_lo=40, ctx_hi=900,
             mix=11, L=1, Hkv=4, D=128, page=64, dtype="bf16", tree=False, ends=2),
        # the end of a tree round of ten attention layers: the accepted paths move together
        dict(name="commit_trees", op="commit", B=64, new_lo=64, new_hi=64, ctx_lo=20, ctx_hi=150,
             mix=12, L=10, Hkv=4, D=128, page=32, dtype="bf16", tree=True, ends=3),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2))) - 1)))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "reserve", "append", "commit"])
    mix = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128, 256])
    if op == "reserve":
        B = _spread(rng, 1, 256)
        lo = rng.choice([1, 4])
        return dict(op=op, B=B, new_lo=lo, new_hi=lo + _spread(rng, 0, 2000), ctx_lo=1,
                    ctx_hi=_spread(rng, 10, 16000), mix=mix, page=page,
                    short=rng.random() < 0.25)
    if op == "append":
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 1, max(1, 16000 // B))
        return dict(op=op, B=B, new_lo=rng.choice([1, max(1, hi // 3)]), new_hi=hi, ctx_lo=0,
                    ctx_hi=_spread(rng, 10, 500), mix=mix, L=rng.choice([1, 1, 2]), Hkv=hkv, D=D,
                    page=page, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "commit":
        tree = rng.random() < 0.6
        T = rng.randint(2, 64)
        return dict(op=op, B=_spread(rng, 1, 64), new_lo=T if tree else 1, new_hi=T, ctx_lo=0,
                    ctx_hi=_spread(rng, 10, 150), mix=mix, L=rng.choice([1, 3, 5]), Hkv=min(hkv, 4),
                    D=min(D, 128), page=page, dtype=rng.choice(["bf16", "bf16", "f32"]), tree=tree,
                    ends=rng.choice([0, 1]))
    group = rng.choice([1, 2, 3, 4, 6, 8])
    form = rng.choice(["token", "drafts", "tree", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    case = dict(op=op, mix=mix, Hq=hkv * group, Hkv=hkv, D=D, page=page, dtype=dtype,
                tree=form == "tree", pad=rng.choice([0, 0, 5]), ctx_lo=rng.choice([0, 100]))
    if form == "token":
        case.update(B=_spread(rng, 1, 64), new_lo=1, new_hi=1, ctx_hi=_spread(rng, 200, 16000))
    elif form == "drafts":
        T = rng.randint(2, 17)
        case.update(B=_spread(rng, 1, 48), new_lo=rng.choice([1, T]), new_hi=T,
                    ctx_hi=_spread(rng, 200, 8000))
    elif form == "tree":
        T = rng.randint(6, 64)
        case.update(B=_spread(rng, 1, 32), new_lo=T, new_hi=T, ctx_hi=_spread(rng, 200, 4000))
    else:
        B = rng.randint(1, 4)
        hi = _spread(rng, 65, 4000 if dtype == "bf16" else 1000)
        case.update(B=B, new_lo=max(1, hi // rng.choice([1, 3, 20])), new_hi=hi,
                    ctx_hi=_spread(rng, 200, 2000))
    return case


def _lengths(case):
    """Cached and new tokens of each sequence: plain lists, from the case alone."""
    r = random.Random(case["mix"])
    ctx = [_spread(r, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [_spread(r, case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return ctx, new


def _trees(case, new):
    """Parents of each sequence's nodes (depth at most 8), from the case alone."""
    r = random.Random(case["mix"] + 1)
    parents, depths = [], []
    for n in new:
        par, dep = [], []
        for v in range(n):
            open_to = [-1] + [u for u in range(v) if dep[u] < 7]
            p = r.choice(open_to[-12:])
            par.append(p)
            dep.append(0 if p < 0 else dep[p] + 1)
        parents.append(par)
        depths.append(dep)
    return parents, depths


def _starts(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def _up(a, b):
    return -(-a // b)


def _i32(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _pool(case, ctx, new, seed, reserved):
    """A page pool in use: every sequence holds the pages of its cached tokens
    (of its new ones too when reserved); the rest is the stack of free pages."""
    page = case["page"]
    r = random.Random(seed)
    have = [_up(c, page) for c in ctx]
    want = [_up(c + n, page) for c, n in zip(ctx, new)]
    need = sum(want) - sum(have)
    n_free = need // 2 if case.get("short") else need + 5
    total = sum(have) + max(n_free, need)
    ids = list(range(total))
    r.shuffle(ids)
    width = max(want) + 1
    table = [[-1] * width for _ in ctx]
    for row, h, w in zip(table, have, want):
        for j in range(w if reserved else h):
            row[j] = ids.pop()
    n_left = len(ids) if reserved else n_free
    # the stack: free pages first, then whatever it held before
    stack = ids + [r.randrange(total) for _ in range(total - len(ids))]
    return dict(n_pages=total, table=_i32(table), free_pages=_i32(stack[:total]), n_left=_i32([n_left]),
                rows=table)


def prepare(case, seed):
    ctx, new = _lengths(case)
    starts = _starts(new)
    N = starts[-1] + case.get("pad", 0)
    pool = _pool(case, ctx, new, seed, reserved=case["op"] != "reserve")
    s = dict(case=case, T=max(new), N=N, n_pages=pool["n_pages"], blocks=pool["table"].shape[1],
             q_start=_i32(starts), seq_len=_i32(ctx), table=pool["table"],
             dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "reserve":
        s.update(free_pages=pool["free_pages"], n_free=pool["n_left"],
                 n_left=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 slots=torch.zeros(N, dtype=torch.int32, device="cuda"))
        return s
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    L, P, H, D, page = case.get("L", 1), pool["n_pages"], case["Hkv"], case["D"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s.update(k_cache=normal(L, P, H, page, D), v_cache=normal(L, P, H, page // 8, D, 8))
    if case["op"] == "attend":
        s.update(q=(1.5 * torch.randn(1, N, case["Hq"], D, generator=g, device="cuda")).to(dt),
                 o=torch.zeros(1, N, case["Hq"], D, device="cuda", dtype=dt), parent=None)
        if case["tree"]:
            # one entry for each of the N rows, of no sequence too
            s["parent"] = _i32(sum(_trees(case, new)[0], []) + [-1] * (N - starts[-1]))
        return s
    slots = [pool["rows"][b][(ctx[b] + i) // page] * page + (ctx[b] + i) % page
             for b in range(case["B"]) for i in range(new[b])]
    s.update(k=normal(L, N, H, D), v=normal(L, N, H, D), slots=_i32(slots))
    if case["op"] == "commit":
        r = random.Random(seed)
        T = s["T"]
        keep, path = [r.randint(0, n) for n in new], None
        if case["tree"]:
            parents = _trees(case, new)[0]
            path = []
            for b, par in enumerate(parents):
                v, way = r.randrange(-1, new[b]), []
                while v >= 0:
                    way.insert(0, v)
                    v = par[v]
                keep[b] = len(way)
                path.append(way + [-1] * (T - len(way)))
        done = [1 if b < case["ends"] and b + 1 < case["B"] else 0 for b in range(case["B"])]
        s.update(n_keep=_i32(keep), path=None if path is None else _i32(path), done=_i32(done),
                 free_pages=pool["free_pages"], n_left=pool["n_left"],
                 n_free=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 seq_len_out=torch.zeros(case["B"], dtype=torch.int32, device="cuda"))
    return s


def _shape(s):
    from speculative_decode_verify_gdn_amd import binding as gb
    c = s["case"]
    return gb.KvShape(L=c.get("L", 1), B=c["B"], Hq=c.get("Hq", c.get("Hkv", 1)), Hkv=c.get("Hkv", 1),
                      D=c.get("D", 128), page=c["page"], n_pages=s["n_pages"], max_blocks=s["blocks"],
                      dtype=DTYPES[c.get("dtype", "bf16")])


def _run_own(s):
    from speculative_decode_verify_gdn_amd import binding as gb
    op = s["case"]["op"]
    if "shape" not in s:  # what a program keeps: its shape, and its workspace
        s["shape"] = _shape(s)
        if op == "attend":
            s["workspace"] = torch.empty(gb.attn_verify_workspace_bytes(s["shape"], s["T"], s["N"]),
                                         dtype=torch.uint8, device="cuda")
    sh = s["shape"]
    if op == "attend":
        gb.attn_verify(sh, s["q"], s["seq_len"], s["table"], s["k_cache"], s["v_cache"], s["o"],
                       s["workspace"], s["T"], q_start=s["q_start"], parent=s["parent"],
                       dev_err=s["dev_err"])
        return s["o"]
    if op == "reserve":
        gb.kv_reserve(sh, s["seq_len"], s["table"], s["free_pages"], s["n_free"], s["n_left"],
                      s["slots"], s["T"], q_start=s["q_start"], dev_err=s["dev_err"])
        return s["slots"], s["table"], s["n_left"]
    if op == "append":
        gb.kv_append(sh, s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                     dev_err=s["dev_err"])
        return s["k_cache"], s["v_cache"]
    gb.kv_commit(sh, s["k"], s["v"], s["slots"], s["n_keep"], s["seq_len"], s["seq_len_out"],
                 s["table"], s["free_pages"], s["n_left"], s["n_free"], s["k_cache"], s["v_cache"],
                 s["T"], q_start=s["q_start"], path=s["path"], done=s["done"], dev_err=s["dev_err"])
    return _committed(s)


def _committed(s):
    out = [s["seq_len_out"], s["free_pages"], s["n_free"]]
    return out + [s["k_cache"], s["v_cache"]] if s["case"]["tree"] else out


def _attend(s):
    c = s["case"]
    B, T, N, Hq, Hkv, D, page = c["B"], s["T"], s["N"], c["Hq"], c["Hkv"], c["D"], c["page"]
    S, G = s["blocks"] * page, Hq // Hkv
    pages = s["table"].long().clamp(min=0)
    k = s["k_cache"][0][pages].float().permute(0, 2, 4, 1, 3).reshape(B, Hkv, D, S)
    v = s["v_cache"][0][pages].float().permute(0, 2, 1, 3, 5, 4).reshape(B, Hkv, S, D)
    first, ctx = s["q_start"][:-1].long(), s["seq_len"].long()
    new = s["q_start"][1:].long() - first
    row = torch.arange(T, device="cuda")
    at = (first[:, None] + row).clamp(max=N - 1)
    q = s["q"][0][at].float().reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    key = torch.arange(S, device="cuda")
    rel = key[None] - ctx[:, None]  # [B,S] place among the new tokens
    if c["tree"]:
        par = s["parent"][:B * T].reshape(B, T).long()
        step = torch.eye(T, device="cuda", dtype=torch.float64) + (par[:, :, None] == row).double()
        above = torch.linalg.matrix_power(step, T) > 0  # an ancestor, or the node itself
        inside = above.gather(2, rel.clamp(0, T - 1)[:, None, :].expand(B, T, S)) & (rel < new[:, None])[:, None]
        live = (rel < 0)[:, None] | inside
    else:
        live = rel[:, None, :] <= row[None, :, None]
    p = torch.matmul(q, k).reshape(B, Hkv, G, T, S) * D ** -0.5
    p.masked_fill_(~live[:, None, None], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(B, Hkv, G * T, S)
    out = torch.matmul(p, v).reshape(B, Hq, T, D).permute(0, 2, 1, 3)
    i = torch.arange(N, device="cuda")
    b = torch.searchsorted(s["q_start"][1:].long(), i, right=True)
    inb = b.clamp(max=B - 1)
    mine = out[inb, (i - first[inb]).clamp(0, T - 1)].to(s["o"].dtype)
    s["o"][0] = torch.where((b < B)[:, None, None], mine, s["o"][0])
    return s["o"]


def _reserve(s):
    c = s["case"]
    page, B = c["page"], c["B"]
    first, ctx = s["q_start"][:-1].long(), s["seq_len"].long()
    new = s["q_start"][1:].long() - first
    have, want = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    need = want - have
    upto = torch.cumsum(need, 0)
    served = (need == 0) | (upto <= s["n_free"])
    j = torch.arange(s["blocks"], device="cuda")[None]
    fresh = served[:, None] & (j >= have[:, None]) & (j < want[:, None])
    src = s["n_free"].long() - 1 - (upto - need)[:, None] - (j - have[:, None])
    got = s["free_pages"][src.clamp(0, s["free_pages"].numel() - 1)]
    s["table"].copy_(torch.where(fresh, got, s["table"]))
    i = torch.arange(s["N"], device="cuda")
    b = torch.searchsorted(s["q_start"][1:].long(), i, right=True).clamp(max=B - 1)
    p = ctx[b] + i - first[b]
    slot = s["table"][b, p // page].long() * page + p % page
    s["slots"].copy_(torch.where(served[b], slot, -1))
    s["n_left"].copy_(s["n_free"] - (need * served).sum())
    return s["slots"], s["table"], s["n_left"]


def _append(s):
    page, slot = s["case"]["page"], s["slots"].long()
    pg, off = slot // page, slot % page
    s["k_cache"][:, pg, :, off] = s["k"].transpose(0, 1)
    s["v_cache"][:, pg, :, off // 8, :, off % 8] = s["v"].transpose(0, 1)
    return s["k_cache"], s["v_cache"]


def _commit(s):
    c = s["case"]
    page, T = c["page"], s["T"]
    first, ctx, keep = s["q_start"][:-1].long(), s["seq_len"].long(), s["n_keep"].long()
    new = s["q_start"][1:].long() - first
    if c["tree"]:
        i = torch.arange(T, device="cuda")
        kept = (i < keep[:, None]).reshape(-1)
        dst = (first[:, None] + i).reshape(-1)
        src = (first[:, None] + s["path"].long().clamp(min=0)).reshape(-1)
        src = torch.where(kept, src, dst)  # a row that is not kept stays as it was written
        slot = s["slots"].long()[dst]
        pg, off = slot // page, slot % page
        sel = kept[:, None, None, None]
        old_k = s["k_cache"][:, pg, :, off]
        old_v = s["v_cache"][:, pg, :, off // 8, :, off % 8]
        s["k_cache"][:, pg, :, off] = torch.where(sel, s["k"].transpose(0, 1)[src], old_k)
        s["v_cache"][:, pg, :, off // 8, :, off % 8] = torch.where(sel, s["v"].transpose(0, 1)[src], old_v)
    length = torch.where(s["done"] != 0, 0, ctx + keep)
    s["seq_len_out"].copy_(length)
    had, left = (ctx + new + page - 1) // page, (length + page - 1) // page
    back = had - left
    j = torch.arange(s["blocks"], device="cuda")[None]
    freed = (j >= left[:, None]) & (j < had[:, None])
    P = s["free_pages"].numel()
    to = torch.where(freed, s["n_left"].long() + (torch.cumsum(back, 0) - back)[:, None] + j - left[:, None], P)
    stack = torch.cat([s["free_pages"], s["free_pages"][:1]])
    stack[to.reshape(-1)] = s["table"].reshape(-1)
    s["free_pages"].copy_(stack[:P])
    s["n_free"].copy_(s["n_left"] + back.sum())
    return _committed(s)


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _attend, "reserve": _reserve, "append": _append, "commit": _commit}[
        state["case"]["op"]](state)


def work(case):
    ctx, new = _lengths(case)
    page, N, B = case["page"], sum(new), case["B"]
    have = sum(_up(c, page) for c in ctx)
    want = sum(_up(c + n, page) for c, n in zip(ctx, new))
    if case["op"] == "reserve":
        return {"bytes": 4 * (2 * B + 1 + 2 * (want - have) + N), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    row = case["Hkv"] * case["D"] * size * 2  # keys and values of one token
    if case["op"] == "append":
        return {"bytes": case["L"] * 2 * N * row + 4 * N, "flops": 0}
    if case["op"] == "commit":
        moved = 0
        if case["tree"]:  # about the mean depth of a node, read and written
            depths = _trees(case, new)[1]
            moved = sum(sum(d) / max(1, len(d)) for d in depths)
        return {"bytes": int(case["L"] * 2 * moved * row) + 4 * (4 * B + 2 * (want - have)), "flops": 0}
    pairs = 0
    if case["tree"]:
        for c, n, d in zip(ctx, new, _trees(case, new)[1]):
            pairs += n * c + sum(x + 1 for x in d)
    else:
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    q = 2 * N * case["Hq"] * case["D"] * size
    return {"bytes": sum(c + n for c, n in zip(ctx, new)) * row + q + 4 * want,
            "flops": 4 * pairs * case["Hq"] * case["D"]}


def exact(case, seed):
    """Written from the definition, one sequence and key head at a time."""
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    starts, page = _starts(new), case["page"]
    if case["op"] == "reserve":
        return None
    if case["op"] == "attend":
        o = s["o"].double()
        G, D = case["Hq"] // case["Hkv"], case["D"]
        parents = _trees(case, new)[0] if case["tree"] else None
        table = s["table"].tolist()
        for b in range(case["B"]):
            total, n, at = ctx[b] + new[b], new[b], starts[b]
            if parents is None:
                hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            else:
                seen = [[False] * n for _ in range(n)]
                for v in range(n):
                    u = v
                    while u >= 0:
                        seen[v][u] = True
                        u = parents[b][u]
                hidden = ~torch.tensor(seen, device="cuda")
            for h in range(case["Hkv"]):
                pages = table[b][:_up(total, page)]
                k = torch.cat([s["k_cache"][0, p, h].double() for p in pages])[:total]
                v = torch.cat([s["v_cache"][0, p, h].double().transpose(1, 2).reshape(page, D)
                               for p in pages])[:total]
                for g in range(G):
                    z = s["q"][0, at:at + n, h * G + g].double() @ k.t() / math.sqrt(D)
                    z[:, ctx[b]:][hidden] = -math.inf
                    o[0, at:at + n, h * G + g] = torch.softmax(z, -1) @ v
        return o
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    slots = s["slots"].tolist()
    keep = range(0)
    if case["op"] == "append":
        pairs = [(t, t) for t in range(len(slots))]
    elif case["tree"]:
        keep, path = s["n_keep"].tolist(), s["path"].tolist()
        pairs = [(starts[b] + i, starts[b] + path[b][i]) for b in range(case["B"]) for i in range(keep[b])]
    else:
        return None
    if len(pairs) > 0:
        to = torch.tensor([slots[d] for d, _ in pairs], device="cuda")
        src = torch.tensor([f for _, f in pairs], device="cuda")
        rows_k, rows_v = s["k"][:, src].double(), s["v"][:, src].double()
        for h in range(case["Hkv"]):
            k_cache[:, to // page, h, to % page] = rows_k[:, :, h]
            for e in range(8):
                mine = (to % 8 == e).nonzero()[:, 0]
                v_cache[:, to[mine] // page, h, to[mine] % page // 8, :, e] = rows_v[:, mine, h]
    if case["op"] == "append":
        return k_cache, v_cache
    return None, None, None, k_cache, v_cache
