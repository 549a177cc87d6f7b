"""Measured cases of the serving operators: attention over a paged 8-bit cache, writing rows into it, and
forking, freeing and compacting its pages.

A cache row is 512 e4m3 values; the rows of a scale block share one fp32 scale. Position p of sequence b is row
p % page_size of page table[b, p // page_size]. With ``own`` false, ``run`` computes the operators with elementary
torch operations in 32 bits; with ``own`` true it calls the package.
"""

import math

import torch

own = False

D = 512
E4M3_MAX = 448.0
E4M3_NAN = 0x7F


# ----------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short conversation: latency counts
        dict(name="attend_one", op="attend", B=1, new=1, L=777, H=64, K=0, page=64, block=64, sink=True),
        # a batch of ordinary conversations, few heads a rank (tensor-parallel serving)
        dict(name="attend_h16", op="attend", B=96, new=1, L=6001, H=16, K=0, page=64, block=32, sink=True),
        # a full serving batch, ragged lengths
        dict(name="attend_h64", op="attend", B=128, new=1, L=5120, H=64, K=0, page=64, block=64, sink=True),
        # few long documents, all heads on one card
        dict(name="attend_long_h128", op="attend", B=3, new=1, L=81920, H=128, K=0, page=128, block=64, sink=False),
        # drafted tokens being verified, four a sequence, small pages
        dict(name="attend_draft", op="attend", B=16, new=4, L=2500, H=32, K=0, page=16, block=16, sink=True),
        # selected rows (window and picks), one token
        dict(name="topk_one", op="attend", B=1, new=1, L=30000, H=128, K=512, page=64, block=64, sink=True),
        # selected rows, a full batch
        dict(name="topk_batch", op="attend", B=256, new=1, L=4096, H=128, K=512, page=64, block=64, sink=True),
        # one new token a sequence
        dict(name="write_token", op="write", B=128, n=1, L=3001, page=64, block=64),
        # whole prompts, ragged
        dict(name="write_prompt", op="write", B=24, n=4096, L=5000, page=64, block=64),
        # four answers from each of a few prompts, and the last ones given back
        dict(name="fork_few", op="fork", B=8, children=32, L=1500, page=64, block=64, pool=4096),
        # beam search over a full batch in a large pool
        dict(name="fork_beams", op="fork", B=128, children=1024, L=2047, page=64, block=32, pool=40000),
        # a pool with holes, its last pages moved to the front
        dict(name="compact_pool", op="compact", B=256, L=4096, page=64, block=64, pool=40000, holes=0.2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128, 256])
    block = rng.choice([b for b in (16, 32, 64) if b <= page])
    op = rng.choice(["attend", "attend", "topk", "topk", "write", "fork", "compact"])
    if op in ("attend", "topk"):
        H = 16 * rng.randint(1, 8)
        L = _log_int(rng, 1, 81920)
        new = rng.choice([1, 1, 1, 2, 3]) if L > 3 else 1
        B = _log_int(rng, 1, max(1, min(300, (1 << 25) // (H * L * new), (1 << 19) // L)))
        K = 0 if op == "attend" else _log_int(rng, 1, 700)
        return dict(op="attend", B=B, new=new, L=L, H=H, K=K, page=page, block=block, sink=rng.random() < 0.6)
    if op == "write":
        n = _log_int(rng, 1, 4096)
        return dict(op="write", B=_log_int(rng, 1, max(1, min(300, 65536 // n))), n=n, L=n + rng.randint(0, 500),
                    page=page, block=block)
    L = _log_int(rng, 20, 4096)
    B = _log_int(rng, 1, max(1, min(256, 400000 // L)))
    if op == "fork":
        c = _log_int(rng, 1, 800)
        return dict(op="fork", B=B, children=c, L=L, page=page, block=block,
                    pool=B * -(-L // page) + c + rng.randint(1, 2000))
    return dict(op="compact", B=B, L=L, page=page, block=block, pool=2 * B * -(-L // page) + rng.randint(1, 2000),
                holes=round(rng.uniform(0.02, 0.6), 3))


def _lens(case):
    """Lengths of the B sequences: the first has L, the others are spread over [L/2, L] (after a write: the rows
    written at least)."""
    L = case["L"]
    lens = [L if i == 0 else max(1, L - (i * 7919) % (L // 2 + 1)) for i in range(case["B"])]
    return [max(x, c) for x, c in zip(lens, _counts(case))] if case["op"] == "write" else lens


def _counts(case):
    """Rows written to each sequence by a write case: the first n, the others spread over [n/2, n]."""
    n = case["n"]
    return [n if i == 0 else max(1, n - (i * 104729) % (n // 2 + 1)) for i in range(case["B"])]


def work(case):
    lens = _lens(case)
    scale_bytes = 4.0 / case["block"]
    page_bytes = case["page"] * (D + scale_bytes)
    pages = sum(-(-x // case["page"]) for x in lens)
    if case["op"] == "attend":
        T, H, K = case["B"] * case["new"], case["H"], case["K"]
        seen = [max(1, x - case["new"] + 1 + i) for x in lens for i in range(case["new"])]
        if K:
            pairs = sum(min(K, x) for x in seen)
            rows = min(pairs, sum(lens))
        else:
            pairs, rows = sum(seen), sum(lens)
        return {"bytes": rows * (D + scale_bytes) + T * H * (4 * D + 4) + 4 * pages + 4 * T * K,
                "flops": 4.0 * D * H * pairs}
    if case["op"] == "write":
        counts = _counts(case)
        earlier = sum((x - c) % case["block"] for x, c in zip(lens, counts))
        return {"bytes": sum(counts) * (3.0 * D + scale_bytes) + 2.0 * earlier * D, "flops": 2.0 * D * sum(counts)}
    if case["op"] == "fork":
        parents = [lens[i % case["B"]] for i in range(case["children"])]
        tails = sum(x % case["page"] > 0 for x in parents)
        entries = sum(-(-x // case["page"]) for x in parents)
        # each shared entry: read, written, given back; its count raised and lowered; the copied last pages
        return {"bytes": 2.0 * tails * page_bytes + entries * 4.0 * 4 + 4.0 * case["pool"], "flops": 0.0}
    live = max(1, round(pages * (1 - case["holes"])))
    # pages of the pool in use lie anywhere, so those behind the first `live` move
    moved = live * (1 - live / case["pool"])
    return {"bytes": 2.0 * moved * page_bytes + 8.0 * case["pool"] + 8.0 * pages, "flops": 0.0}


# ----------------------------------------------------------------------------------------------------- inputs
def _pow2_scale(amax):
    """The least power of two s >= 2^-100 with amax <= 448 s, elementwise (32-bit, exact)."""
    m, x = torch.frexp(amax.float())                       # amax = m 2^x, m in [0.5, 1)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(min=-100)
    e = torch.where(amax > 0, e, torch.full_like(e, -100))
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _to_codes(y):
    """Bytes of the e4m3 values nearest to y (ties to even), saturated."""
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _from_codes(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32)


def _fill_pool(gen, pool, page, block, dev):
    """Pages full of N(0,1) rows at their blocks' scales."""
    codes = torch.empty(pool, page, D, dtype=torch.uint8, device=dev)
    scales = torch.empty(pool, page // block, dtype=torch.float32, device=dev)
    x = torch.randn(pool, page // block, block * D, generator=gen, device=dev)
    scales.copy_(_pow2_scale(x.abs().amax(dim=2)))
    codes.copy_(_to_codes(x / scales[:, :, None]).view(pool, page, D))
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    page, block, B = case["page"], case["block"], case["B"]
    lens = _lens(case)
    used = [-(-x // page) for x in lens]
    width = max(used) + 1
    pool = case.get("pool", sum(used) + 3)
    codes, scales = _fill_pool(gen, pool, page, block, dev)
    # pages in no order, as after hours of serving
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    n_used = torch.tensor(used, device=dev)
    slots = torch.arange(width, device=dev)
    inside = slots < n_used[:, None]
    first = torch.cumsum(n_used, 0) - n_used
    table = torch.where(inside, order[(first[:, None] + slots).clamp(max=pool - 1)], -1).to(torch.int32)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)
    # rows behind the last one of a sequence hold whatever was there
    last = table.gather(1, (n_used - 1)[:, None])[:, 0].long()
    behind = torch.arange(page, device=dev) >= ((lens_t - 1) % page + 1)[:, None]
    codes[last] = torch.where(behind[:, :, None], E4M3_NAN, codes[last])
    refcount = torch.zeros(pool, dtype=torch.int32, device=dev)
    refcount[order[: sum(used)].long()] = 1
    state = dict(case=dict(case), codes=codes, scales=scales, table=table, lens=lens_t, refcount=refcount)

    if case["op"] == "attend":
        T, H, K, new = B * case["new"], case["H"], case["K"], case["new"]
        state["q"] = torch.randn(T, H, D, generator=gen, device=dev).to(torch.bfloat16)
        state["sink"] = torch.randn(H, generator=gen, device=dev) if case["sink"] else None
        state["seq"] = torch.arange(B, device=dev, dtype=torch.int32).repeat_interleave(new)
        seen = lens_t[:, None] - new + 1 + torch.arange(new, device=dev, dtype=torch.int32)
        state["seen"] = seen.clamp(min=1).reshape(-1).to(torch.int32)
        if K:
            # the last rows and picks of the others, all different; -1 where a sequence has fewer
            vis = state["seen"][:, None].long()
            keys = torch.rand(T, max(K, max(lens)), generator=gen, device=dev)
            pos = torch.arange(keys.shape[1], device=dev)
            keys = torch.where(pos >= vis - min(128, K // 4), keys + 1.0, keys)
            keys = torch.where(pos < vis, keys, -1.0)
            top, picks = torch.topk(keys, K, dim=1)
            state["topk"] = torch.where(top >= 0, picks, -1).to(torch.int32)
    elif case["op"] == "write":
        counts = _counts(case)
        n = torch.tensor(counts, dtype=torch.int32, device=dev)
        state["cu"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), torch.cumsum(n, 0).to(torch.int32)])
        state["start"] = lens_t - n
        # larger by up to twice than what the blocks hold, so that some scales grow
        loud = 0.5 + 1.5 * torch.rand(sum(counts), 1, generator=gen, device=dev)
        state["rows"] = (torch.randn(sum(counts), D, generator=gen, device=dev) * loud).to(torch.bfloat16)
    elif case["op"] == "fork":
        state["parents"] = (torch.arange(case["children"], device=dev, dtype=torch.int32) % B).to(torch.int32)
        state["children"] = torch.full((case["children"], width), -1, dtype=torch.int32, device=dev)
    else:
        gone = torch.rand(B, width, generator=gen, device=dev) < case["holes"]
        dead = table[gone & inside].long()
        refcount[dead] = 0
        state["table"] = torch.where(gone, -1, table).to(torch.int32)
    return state


# ----------------------------------------------------------------------------------------------------- plain forms
def _attend_plain(s):
    case = s["case"]
    page, block, K = case["page"], case["block"], case["K"]
    table = s["table"][s["seq"].long()].long()
    seen = s["seen"][:, None].long()
    pos = s["topk"].long() if K else torch.arange(case["L"], device=seen.device)[None, :].expand(seen.shape[0], -1)
    ok = (pos >= 0) & (pos < seen)
    at = torch.where(ok, pos, 0)
    row = table.gather(1, at // page).clamp(min=0) * page + at % page
    kv = _from_codes(s["codes"].view(-1, D)[row]) * s["scales"].view(-1)[row // block][:, :, None]
    kv = torch.where(ok[:, :, None], kv, 0.0)
    sc = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * (1.0 / math.sqrt(D))
    sc = torch.where(ok[:, None, :], sc, -math.inf)
    m = sc.amax(dim=2, keepdim=True)
    if s["sink"] is not None:
        m = torch.maximum(m, s["sink"][None, :, None])
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m)
    total = p.sum(dim=2, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(s["sink"][None, :, None] - m)
    o = torch.matmul(p, kv) / torch.where(total > 0, total, 1.0)
    return o.to(torch.bfloat16), (m + torch.log(total))[:, :, 0]


def _write_plain(s):
    case = s["case"]
    page, block = case["page"], case["block"]
    rows, cu, start, codes, scales = s["rows"], s["cu"].long(), s["start"].long(), s["codes"], s["scales"]
    flat, fs = codes.view(-1, D), scales.view(-1)
    i = torch.arange(rows.shape[0], device=rows.device)
    b = torch.searchsorted(cu, i, right=True) - 1
    p = start[b] + i - cu[b]
    row = s["table"].long()[b, p // page] * page + p % page
    x = rows.float()
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=1)
    top = torch.zeros_like(fs).scatter_reduce_(0, row // block, amax, "amax")
    need = _pow2_scale(top)
    touched = torch.zeros_like(fs).index_fill_(0, row // block, 1.0) > 0
    # the block that a sequence's first new row goes to may hold earlier rows
    lead = row[cu[:-1]] // block
    kept = start % block
    old = fs[lead]
    grown = torch.where(kept > 0, torch.maximum(old, need[lead]), need[lead])
    new = torch.where(touched, need, fs)
    new[lead] = grown
    at = torch.arange(block, device=rows.device)
    earlier = flat.view(-1, block, D)[lead]
    again = _to_codes(_from_codes(earlier) * (old / grown)[:, None, None])
    flat.view(-1, block, D)[lead] = torch.where((at < kept[:, None])[:, :, None], again, earlier)
    flat[row] = _to_codes(x / new[row // block][:, None])
    fs.copy_(new)


def _free_plain(table, refcount):
    refcount.scatter_add_(0, table.clamp(min=0).long().view(-1), -(table >= 0).to(torch.int32).view(-1))
    table.fill_(-1)


def _fork_plain(s):
    page, codes, scales, refcount = s["case"]["page"], s["codes"], s["scales"], s["refcount"]
    rows, n = s["table"][s["parents"].long()].long(), s["lens"][s["parents"].long()].long()
    full = n // page
    slots = torch.arange(rows.shape[1], device=rows.device)
    share = slots < full[:, None]
    refcount.scatter_add_(0, rows.clamp(min=0).view(-1), share.to(torch.int32).view(-1))
    tail = n % page > 0
    free = torch.argsort((refcount > 0).to(torch.int8), stable=True)
    fresh = free[(torch.cumsum(tail, 0) - 1).clamp(min=0)]
    src = rows.gather(1, full.clamp(max=rows.shape[1] - 1)[:, None])[:, 0]
    src, dst = src[tail], fresh[tail]
    codes[dst] = codes[src]
    scales[dst] = scales[src]
    refcount[dst] = 1
    child = torch.where(share, rows, -1)
    child = torch.where((slots == full[:, None]) & tail[:, None], fresh[:, None], child)
    s["children"].copy_(child)


def _compact_plain(s):
    codes, scales, refcount, table = s["codes"], s["scales"], s["refcount"], s["table"].long()
    live = refcount > 0
    n = live.sum()
    index = torch.arange(live.shape[0], device=live.device)
    src = (live & (index >= n)).nonzero()[:, 0]
    dst = (~live & (index < n)).nonzero()[:, 0]
    codes[dst] = codes[src]
    scales[dst] = scales[src]
    count = refcount.clone()
    count[dst] = refcount[src]
    count[src] = 0
    to = index.clone()
    to[src] = dst
    return torch.where(table >= 0, to[table.clamp(min=0)], -1).to(torch.int32), count


# ----------------------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        import sparse_mla_attention_gb300 as smla
        if "cache" not in s:      # the handle and workspace that a program keeps
            s["cache"] = smla.PagedCache(s["codes"].view(torch.float8_e4m3fn), s["scales"], s["refcount"])
            s["workspace"] = smla.Workspace(s["codes"].device)
        cache, ws = s["cache"], s["workspace"]
        if case["op"] == "attend":
            return smla.sparse_mla_fwd_paged(s["q"], cache, s["table"], s["seen"], topk=s.get("topk"), seq=s["seq"],
                                             sink=s["sink"], workspace=ws, check_status=False)
        if case["op"] == "write":
            smla.cache_write(cache, s["table"], s["start"], s["cu"], s["rows"], workspace=ws, check_status=False)
        elif case["op"] == "fork":
            smla.cache_free(cache, s["children"], workspace=ws, check_status=False)
            smla.cache_fork(cache, s["table"], s["lens"], s["parents"], out=s["children"], workspace=ws,
                            check_status=False)
        else:
            table, count = smla.cache_compact(cache, s["table"], workspace=ws, check_status=False)
    else:
        if case["op"] == "attend":
            return _attend_plain(s)
        if case["op"] == "write":
            _write_plain(s)
        elif case["op"] == "fork":
            _free_plain(s["children"], s["refcount"])
            _fork_plain(s)
        else:
            table, count = _compact_plain(s)
    values = s["codes"].view(torch.float8_e4m3fn)
    if case["op"] == "write":
        return values, s["scales"]
    if case["op"] == "fork":
        return s["children"], s["refcount"], values, s["scales"]
    return table, count, values, s["scales"]


# ----------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    page, block = case["page"], case["block"]
    codes, scales = s["codes"], s["scales"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    if case["op"] == "attend":
        outs, lses = [], []
        seq, seen = s["seq"].tolist(), s["seen"].tolist()
        for t in range(len(seq)):
            if case["K"]:
                at = s["topk"][t].long()
                at = at[(at >= 0) & (at < seen[t])]
            else:
                at = torch.arange(seen[t], device=codes.device)
            where = s["table"][seq[t]].long()
            x = codes[where[at // page], at % page].view(torch.float8_e4m3fn).to(torch.float64)
            x = x * scales[where[at // page], (at % page) // block].double()[:, None]
            logits = (s["q"][t].double() @ x.T) / math.sqrt(512.0)
            if s["sink"] is not None:
                logits = torch.cat([logits, s["sink"].double()[:, None]], dim=1)
            lse = torch.logsumexp(logits, dim=1)
            outs.append(torch.exp(logits[:, : x.shape[0]] - lse[:, None]) @ x)
            lses.append(lse)
        return torch.stack(outs), torch.stack(lses)
    if case["op"] == "write":
        cu, start = s["cu"].tolist(), s["start"].tolist()

        def nearest(y):
            # e4m3: 4 significant bits, spacing 2^-9 at the least (the exponent's bits alone are a power of two)
            power = y.abs().clamp(min=2.0 ** -6).contiguous().view(torch.int64) >> 52 << 52
            gap = power.view(torch.float64) / 8.0
            return torch.round(y / gap) * gap
        values = codes.view(torch.float8_e4m3fn).to(torch.float64)
        out_scales = scales.double()
        for b in range(len(start)):
            done, end = start[b], start[b] + cu[b + 1] - cu[b]
            while done < end:
                upto = min(end, (done // block + 1) * block)
                pg, lo = table[b][done // page], done % page
                k, kept = lo // block, lo % block
                x = s["rows"][cu[b] + done - start[b]: cu[b] + upto - start[b]].double()
                big = float(x.abs().max())
                e = max(-100, math.ceil(math.log2(big / 448.0))) if big > 0 else -100
                while 448.0 * 2.0 ** e < big:
                    e += 1
                while e > -100 and 448.0 * 2.0 ** (e - 1) >= big:
                    e -= 1
                sc = 2.0 ** e
                if kept:
                    was = float(out_scales[pg, k])
                    sc = max(sc, was)
                    head = slice(k * block, k * block + kept)
                    values[pg, head] = nearest(values[pg, head] * (was / sc))
                out_scales[pg, k] = sc
                values[pg, lo: lo + upto - done] = nearest(x / sc)
                done = upto
        return values, out_scales
    values = codes.view(torch.float8_e4m3fn).to(torch.float64)
    moved = scales.double()
    if case["op"] == "fork":
        count, width = s["refcount"].tolist(), len(table[0])
        free = [i for i, c in enumerate(count) if c == 0]
        kids = []
        for p in s["parents"].tolist():
            row = [-1] * width
            whole, rest = divmod(lens[p], page)
            for j in range(whole):
                row[j] = table[p][j]
                count[row[j]] += 1
            if rest:
                row[whole] = free.pop(0)
                count[row[whole]] = 1
                values[row[whole]] = values[table[p][whole]]
                moved[row[whole]] = moved[table[p][whole]]
            kids.append(row)
        return torch.tensor(kids), torch.tensor(count), values, moved
    count = s["refcount"].tolist()
    n = sum(c > 0 for c in count)
    src = [i for i, c in enumerate(count) if c > 0 and i >= n]
    dst = [i for i, c in enumerate(count) if c == 0 and i < n]
    for a, b in zip(src, dst):
        count[b], count[a] = count[a], 0
    to = dict(zip(src, dst))
    if src:
        values[dst] = values[src]
        moved[dst] = moved[src]
    return torch.tensor([[to.get(v, v) for v in row] for row in table]), torch.tensor(count), values, moved
