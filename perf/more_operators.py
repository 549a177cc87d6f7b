"""Measured cases of what a decode loop does with the paged 8-bit cache besides attending to it: accumulating the
attention weight that each cached position gets, evicting the positions that got least, choosing the next beams over the
vocabulary, and reordering the cache's sequences after that choice.

The cache is that of perf/operators.py: a row is 512 e4m3 values, the rows of a scale block share one fp32 scale, and
position p of sequence b is row p % page_size of page table[b, p // page_size]. With ``own`` false, ``run`` computes the
operators with elementary torch operations (32 bits, 64 where two candidates' order hangs on it); with ``own`` true it
calls the package.
"""

import math
import random

import torch

own = False

D = 512


# ----------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short conversation, after each token: latency counts
        dict(name="watch_one", op="watch", B=1, new=1, L=777, H=64, page=64, block=64, decay=1.0),
        # a batch of ordinary conversations, few heads a rank (tensor-parallel serving)
        dict(name="watch_h16", op="watch", B=96, new=1, L=6001, H=16, page=64, block=32, decay=0.9),
        # a full serving batch, ragged lengths
        dict(name="watch_h64", op="watch", B=128, new=1, L=5120, H=64, page=64, block=64, decay=1.0),
        # the last tokens of long prompts vote on what to keep of them, all heads on one card
        dict(name="watch_prompt", op="watch", B=4, new=32, L=20000, H=128, page=128, block=64, decay=0.0),
        # one conversation at its budget
        dict(name="evict_one", op="evict", B=1, L=1500, keep=1024, first=4, recent=256, page=64, block=64, spare=64),
        # a full batch brought back to its budget
        dict(name="evict_batch", op="evict", B=64, L=8192, keep=2048, first=16, recent=512, page=64, block=64,
             spare=100),
        # long documents, after their prompts
        dict(name="evict_long", op="evict", B=3, L=81920, keep=16384, first=0, recent=64, page=128, block=32,
             spare=1000),
        # one request, four beams, logits in 32 bits
        dict(name="select_one", op="select", B=1, K=4, n=4, V=32000, dtype="float32", pad=0, done=False, ban=0.0),
        # odd sizes: twice as many candidates as beams are kept, rows that start anywhere, banned tokens
        dict(name="select_odd", op="select", B=7, K=5, n=10, V=50001, dtype="float16", pad=0, done=True, ban=0.3),
        # a full batch over a large vocabulary
        dict(name="select_batch", op="select", B=32, K=8, n=8, V=128000, dtype="bfloat16", pad=128, done=True, ban=0.0),
        # eight requests of four beams
        dict(name="reorder_few", op="reorder", B=8, K=4, L=1500, page=64, block=64, pool=4096, weights=False),
        # beam search over a full batch in a large pool, with the accumulated weights
        dict(name="reorder_beams", op="reorder", B=128, K=8, L=2047, page=64, block=32, pool=40000, weights=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128, 256])
    block = rng.choice([b for b in (16, 32, 64) if b <= page])
    op = rng.choice(["watch", "watch", "evict", "select", "select", "reorder"])
    if op == "watch":
        H = 16 * rng.randint(1, 8)
        L = _log_int(rng, 1, 81920)
        new = min(L, rng.choice([1, 1, 1, 2, 5, 32]))
        B = _log_int(rng, 1, max(1, min(300, (1 << 28) // (H * L * new), (1 << 19) // L)))
        return dict(op=op, B=B, new=new, L=L, H=H, page=page, block=block, decay=rng.choice([0.0, 0.9, 1.0]))
    if op == "evict":
        L = _log_int(rng, 2, 81920)
        keep = rng.randint(1, L)
        first = rng.randint(0, min(64, keep))
        recent = rng.randint(0, keep - first)
        return dict(op=op, B=_log_int(rng, 1, max(1, min(300, (1 << 17) // L))), L=L, keep=keep, first=first,
                    recent=recent, page=page, block=block, spare=rng.randint(0, 300))
    if op == "select":
        V = _log_int(rng, 20, 140000)
        K = _log_int(rng, 1, 16)
        n = min(64, K * V, rng.choice([K, K, 2 * K, rng.randint(1, 64)]))
        return dict(op=op, B=_log_int(rng, 1, max(1, min(300, (1 << 24) // (K * V)))), K=K, n=n, V=V,
                    dtype=rng.choice(["float32", "float16", "bfloat16"]), pad=rng.choice([0, 0, 1, 64]),
                    done=rng.random() < 0.5, ban=rng.choice([0.0, 0.0, 0.2]))
    K = rng.randint(1, 10)
    L = _log_int(rng, 1, 4096)
    B = _log_int(rng, 1, max(1, min(128, 250000 // (L * K))))
    return dict(op=op, B=B, K=K, L=L, page=page, block=block, pool=2 * B * K * -(-L // page) + rng.randint(1, 2000),
                weights=rng.random() < 0.5)


def _lens(case):
    """Lengths of the sequences (of the groups of beams): the first has L, the others are spread over [L/2, L]."""
    L = case["L"]
    return [L if i == 0 else max(1, L - (i * 7919) % (L // 2 + 1)) for i in range(case["B"])]


def _tokens(case):
    """New tokens of each sequence: the first has all of them, the others at least half, none more than its length."""
    new = case["new"]
    return [min(x, new if i == 0 else max(1, new - (i * 13) % (new // 2 + 1))) for i, x in enumerate(_lens(case))]


def _width(case):
    return -(-case["L"] // case["page"]) + 1


def work(case):
    if case["op"] == "select":
        rows = case["B"] * case["K"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": rows * (case["V"] * size + 5) + case["B"] * case["n"] * 12, "flops": 3.0 * rows * case["V"]}
    lens = _lens(case)
    row = D + 4.0 / case["block"]
    pages = sum(-(-x // case["page"]) for x in lens)
    if case["op"] == "watch":
        new = _tokens(case)
        pairs = sum(n * x - n * (n - 1) // 2 for n, x in zip(new, lens))
        once = 4 if case["decay"] == 0.0 else 8
        return {"bytes": sum(lens) * (row + once) + sum(new) * (case["H"] * (2 * D + 4) + 4) + 4 * pages,
                "flops": (2.0 * D + 4) * case["H"] * pairs}
    width = _width(case)
    if case["op"] == "evict":
        kept = sum(min(x, case["keep"]) for x in lens)
        table = case["B"] * (4 * width + 4)
        return {"bytes": 2 * kept * row + 4 * sum(lens) + 4 * case["B"] * (width * case["page"] + case["keep"])
                + 4 * pages + table, "flops": 0}
    rows = case["B"] * case["K"]
    copies = [len(k) - len(set(k)) for k in _kids(case)]
    moved = sum(c * (x % case["page"]) for c, x in zip(copies, lens))
    state = 4 * case["K"] * sum(x + width * case["page"] for x in lens) if case["weights"] else 0
    return {"bytes": 2 * moved * row + rows * (8 * width + 12) + state, "flops": 0}


# ----------------------------------------------------------------------------------------------------- inputs
def _kids(case):
    """Which beam of its group each new beam continues (as beams do: the best go on several times, others end)."""
    rng, K = random.Random(case["B"] * 1000 + case["K"]), case["K"]
    return [rng.choices(range(K), [0.75 ** k for k in range(K)], k=K) for _ in range(case["B"])]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _randn(g, *size):
    return torch.randn(*size, generator=g, device="cuda")


def _pool(case, g, num_pages):
    """Pages of N(0,1) rows in e4m3 with block scales of 2^-8 to 2^-5 (each block's rows of its own size)."""
    page, blocks = case["page"], case["page"] // case["block"]
    scales = torch.exp2(-torch.randint(5, 9, (num_pages, blocks), generator=g, device="cuda").float())
    codes = torch.empty(num_pages, page, D, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (page * D))
    for i in range(0, num_pages, step):
        part = _randn(g, min(step, num_pages - i), page, D) * 64.0
        codes[i:i + step] = part.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _place(case, g, num_pages, lens):
    """Block table with pages of the pool, in any order, for sequences of these lengths."""
    width = _width(case)
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    need = torch.tensor([-(-x // case["page"]) for x in lens], device="cuda")
    start = torch.cumsum(need, 0) - need
    j = torch.arange(width, device="cuda")
    at = (start[:, None] + j).clamp(max=num_pages - 1)
    return torch.where(j < need[:, None], order[at], -1).contiguous(), int(need.sum()), order


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "select":
        rows, V = case["B"] * case["K"], case["V"]
        logits = _randn(g, rows, V + case["pad"]) * 3.0
        if case["ban"]:
            logits[torch.rand(logits.shape, generator=g, device="cuda") < case["ban"]] = -math.inf
        scores = -_randn(g, case["B"], case["K"]).abs() * 4.0
        done = (torch.rand(case["B"], case["K"], generator=g, device="cuda") < 0.2) if case["done"] else None
        return dict(case=case, logits=logits.to(getattr(torch, case["dtype"]))[:, :V], scores=scores, done=done,
                    eos=V // 2)
    lens = _lens(case)
    s = dict(case=case)
    page, width = case["page"], _width(case)
    if case["op"] == "reorder":
        return _prepare_reorder(case, g, lens, s)
    pages = sum(-(-x // page) for x in lens)
    extra = sum(-(-min(x, case["keep"]) // page) for x in lens) + case["spare"] if case["op"] == "evict" else 3
    s["codes"], s["scales"] = _pool(case, g, pages + extra)
    s["table"], used, order = _place(case, g, pages + extra, lens)
    s["refcount"] = torch.zeros(pages + extra, dtype=torch.int32, device="cuda")
    s["refcount"][order[:used].long()] = 1
    if case["op"] == "evict":
        s["lens"] = _i32(lens)
        # what heads add up to is heavy-tailed; positions that nobody looked at have nothing
        w = torch.exp(2.0 * _randn(g, case["B"], width * page))
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, 0.0, w)
        s["new_table"] = torch.full_like(s["table"], -1)
        s["new_lens"] = torch.zeros_like(s["lens"])
        s["new_weights"] = torch.zeros_like(s["weights"])
        s["kept"] = torch.zeros(case["B"], case["keep"], dtype=torch.int32, device="cuda")
        return s
    new = _tokens(case)
    T, H = sum(new), case["H"]
    s["q"] = (2.0 * _randn(g, T, H, D)).to(torch.bfloat16)
    s["cu"] = _i32([0] + new).cumsum(0).to(torch.int32)
    s["lens"] = _i32([x - n + 1 + i for x, n in zip(lens, new) for i in range(n)])
    s["earlier"] = torch.exp(_randn(g, case["B"], width * page))
    s["out"] = torch.zeros_like(s["earlier"])
    # of the attention that came before, with a sink of weight 1
    lse = torch.empty(T, H, device="cuda")
    at = 0
    for b, n in enumerate(new):
        x = _values(s, s["table"][b:b + 1], lens[b])[0]
        logits = s["q"][at:at + n].float() @ x.T / math.sqrt(D)
        logits.masked_fill_(torch.arange(lens[b], device="cuda") >= s["lens"][at:at + n, None, None], -math.inf)
        lse[at:at + n] = torch.logaddexp(torch.logsumexp(logits, 2), torch.zeros((), device="cuda"))
        at += n
    s["lse"] = lse
    return s


def _prepare_reorder(case, g, lens, s):
    """Groups of K beams: the first half of a group's positions is the prompt, whose full pages its beams share."""
    B, K, page, width = case["B"], case["K"], case["page"], _width(case)
    lens = torch.tensor(lens, device="cuda").repeat_interleave(K)
    shared = (lens // 2) // page
    whole = (lens + page - 1) // page
    own_pages = whole - shared
    lead = torch.arange(B * K, device="cuda") // K * K
    first = torch.arange(B * K, device="cuda") == lead
    takes = own_pages + torch.where(first, shared, 0)
    start = torch.cumsum(takes, 0) - takes
    order = torch.randperm(case["pool"], generator=g, device="cuda")
    j = torch.arange(width, device="cuda")
    mine = start[:, None] + torch.where(first, shared, 0)[:, None] + (j - shared[:, None])
    at = torch.where(j < shared[:, None], start[lead][:, None] + j, mine)
    table = torch.where(j < whole[:, None], order[at.clamp(0, case["pool"] - 1)], -1)
    s["table"] = table.to(torch.int32)
    s["count0"] = torch.bincount(table[table >= 0], minlength=case["pool"]).to(torch.int32)
    s["refcount"] = s["count0"].clone()
    s["lens"] = lens.to(torch.int32)
    s["parents"] = _i32([k + K * i for i, kids in enumerate(_kids(case)) for k in kids])
    s["codes"], s["scales"] = _pool(case, g, case["pool"])
    s["weights"] = torch.exp(_randn(g, B * K, width * page)) if case["weights"] else None
    s["new_table"] = torch.full_like(s["table"], -1)
    s["new_lens"] = torch.zeros_like(s["lens"])
    s["new_weights"] = torch.zeros_like(s["weights"]) if case["weights"] else None
    return s


# ----------------------------------------------------------------------------------------------------- plain forms
def _values(s, table, n):
    """The first n positions of each sequence of `table`, in 32 bits: [B, n, 512]."""
    page, block = s["case"]["page"], s["case"]["block"]
    at = torch.arange(n, device="cuda")
    pages = table[:, at // page].long().clamp(min=0)
    x = s["codes"].view(torch.float8_e4m3fn)[pages, at % page].float()
    return x * s["scales"][pages, at % page // block][..., None]


def _watch_plain(s):
    case = s["case"]
    B, H, L, new = case["B"], case["H"], case["L"], case["new"]
    cu = s["cu"].long()
    i = torch.arange(new, device="cuda")
    there = i < (cu[1:] - cu[:-1])[:, None]
    token = torch.where(there, cu[:-1, None] + i, 0)
    lens = torch.where(there, s["lens"][token], 0)
    x = _values(s, s["table"], L)
    p = torch.matmul(s["q"][token].float().view(B, new * H, D), x.transpose(1, 2)).view(B, new, H, L)
    p = torch.exp(p / math.sqrt(D) - s["lse"][token][..., None])
    seen = torch.arange(L, device="cuda") < lens[..., None]
    p = torch.where(seen[:, :, None], p, 0.0).sum((1, 2))
    if case["decay"]:
        p = p + case["decay"] * s["earlier"][:, :L]
    s["out"][:, :L] = torch.where(seen.any(1), p, s["out"][:, :L])
    return s["out"]


def _rank(x, desc):
    """The order of each row's values, ties by the lowest index."""
    return torch.sort(x, dim=-1, descending=desc, stable=True)[1]


def _evict_plain(s):
    case = s["case"]
    page, block, keep = case["page"], case["block"], case["keep"]
    table, new = s["table"], s["new_table"]
    # the pages of the last pass go back
    count, old = s["refcount"], new[new >= 0].long()
    count.index_put_((old,), torch.full_like(old, -1, dtype=torch.int32), accumulate=True)
    L = s["lens"].long()[:, None]
    at = torch.arange(s["weights"].shape[1], device="cuda")
    w = torch.where((at < case["first"]) | (at >= L - case["recent"]), math.inf, s["weights"])
    w = torch.where(at < L, w, -math.inf)
    kept = _rank(w, True)[:, :keep]
    n = torch.clamp(L, max=keep)
    i = torch.arange(keep, device="cuda")
    kept = torch.sort(torch.where(i < n, kept, 1 << 30))[0]
    there = i < n
    src = torch.where(there, kept, 0)
    # lowest free pages first, sequence after sequence
    need = (n + page - 1) // page
    j = torch.arange(table.shape[1], device="cuda")
    has = j < need
    free = torch.nonzero(count == 0)[:, 0]
    nth = (torch.cumsum(need, 0) - need) + j
    new.copy_(torch.where(has, free[nth.clamp(max=free.shape[0] - 1)], -1))
    count[new[has].long()] = 1
    # rows: a block has the largest scale of what it takes
    pages = torch.gather(table.long(), 1, src // page)
    sc = torch.where(there, s["scales"][pages, src % page // block], 0.0)
    blocks = torch.nn.functional.pad(sc, (0, -keep % block)).view(case["B"], -1, block).amax(2)
    to = torch.gather(new.long(), 1, (i // page).expand_as(src))
    values = s["codes"].view(torch.float8_e4m3fn)
    ratio = sc / blocks.repeat_interleave(block, 1)[:, :keep]
    x = (values[pages, src % page].float() * ratio[..., None]).to(torch.float8_e4m3fn)
    slot = (i % page).expand_as(src)
    s["codes"][to[there], slot[there]] = x.view(torch.uint8)[there]
    lead = there & (i % block == 0)
    s["scales"][to[lead], slot[lead] // block] = blocks.repeat_interleave(block, 1)[:, :keep][lead]
    s["new_weights"].zero_()
    s["new_weights"][:, :keep] = torch.where(there, torch.gather(s["weights"], 1, src), 0.0)
    s["kept"].copy_(torch.where(there, kept, -1))
    s["new_lens"].copy_(n[:, 0])
    return s["new_table"], s["new_lens"], s["new_weights"], s["kept"]


def _select_plain(s):
    case = s["case"]
    B, K, n, V = case["B"], case["K"], case["n"], case["V"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True).double()
    lse = top[:, 0] + torch.log(torch.exp(x.double() - top).sum(1))
    # a row's best n: 64-bit keys of the value's order and, below it, the lowest index first
    bits = x.view(torch.int32).long()
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = (bits << 32) | (0xFFFFFFFF - torch.arange(V, device="cuda"))
    best = torch.topk(key, min(n, V), dim=1)[0]
    token = 0xFFFFFFFF - (best & 0xFFFFFFFF)
    before = s["scores"].view(-1, 1).double()
    score = before + (torch.gather(x, 1, token).double() - lse[:, None])
    if s["done"] is not None:
        over = s["done"].view(-1, 1)
        lone = torch.arange(token.shape[1], device="cuda") == 0
        score = torch.where(over, torch.where(lone, before, -math.inf), score)
        token = torch.where(over, s["eos"], token)
    score = torch.where(torch.isfinite(score), score, -math.inf)
    # the group's best n, ties by beam and token
    m = token.shape[1]
    beam = torch.arange(K, device="cuda").view(K, 1)
    flat = (beam * V + token.view(B, K, m)).view(B, K * m)
    score = score.view(B, K * m)
    by = torch.gather(_rank(flat, False), 1, _rank(torch.gather(score, 1, _rank(flat, False)), True))[:, :n]
    score, flat = torch.gather(score, 1, by), torch.gather(flat, 1, by)
    fine = torch.isfinite(score)
    parent = torch.arange(B, device="cuda").view(B, 1) * K + flat // V
    pad = (0, n - score.shape[1])
    parent, token = torch.where(fine, parent, -1), torch.where(fine, flat % V, -1)
    return (torch.nn.functional.pad(parent, pad, value=-1).int(), torch.nn.functional.pad(token, pad, value=-1).int(),
            torch.nn.functional.pad(torch.where(fine, score, -math.inf), pad, value=-math.inf).float())


def _reorder_plain(s):
    case = s["case"]
    page = case["page"]
    table, lens, parents, count = s["table"], s["lens"].long(), s["parents"].long(), s["refcount"]
    rows, width = table.shape
    j = torch.arange(width, device="cuda")
    kids = torch.bincount(parents, minlength=rows)
    order = torch.arange(rows, device="cuda")
    first = torch.full((rows,), rows, device="cuda").scatter_reduce(0, parents, order, "amin")
    heir = first[parents] == order
    tail = torch.gather(table, 1, (lens // page)[:, None].clamp(max=width - 1))[:, 0].long()
    part = lens % page > 0
    # a further child's copy goes to the last page of a row that ends, else to a free page
    ends = (kids == 0) & part
    ends &= torch.where(ends, count[tail.clamp(min=0)], 0) == 1
    copies = torch.nonzero(~heir & part[parents])[:, 0]
    pages = torch.cat([tail[ends], torch.nonzero(count == 0)[:, 0]])[:copies.shape[0]]
    mine = torch.full((rows,), -1, device="cuda")
    mine[copies] = pages
    line = table[parents].long()
    full = (lens // page)[parents, None]
    line = torch.where(heir[:, None] | (j < full), line, torch.where(j == full, mine[:, None], -1))
    s["new_table"].copy_(line)
    held = line[line >= 0]
    count.copy_(torch.bincount(held, minlength=count.shape[0]))
    s["codes"][pages] = s["codes"][tail[parents[copies]]]
    s["scales"][pages] = s["scales"][tail[parents[copies]]]
    s["new_lens"].copy_(lens[parents])
    if s["weights"] is not None:
        at = torch.arange(s["weights"].shape[1], device="cuda")
        s["new_weights"].copy_(torch.where(at < lens[parents, None], s["weights"][parents], 0.0))


# ----------------------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import sparse_mla_attention_gb300 as smla
        if "workspace" not in s:      # the handle and workspace that a program keeps
            s["workspace"] = smla.Workspace("cuda")
            if op != "select":
                s["cache"] = smla.PagedCache(s["codes"].view(torch.float8_e4m3fn), s["scales"], s["refcount"])
        ws = s["workspace"]
        if op == "select":
            return smla.beam_select(s["logits"], s["scores"], n=case["n"], done=s["done"], eos=s["eos"], workspace=ws)
        cache = s["cache"]
        if op == "watch":
            return smla.cache_weights(s["q"], cache, s["table"], s["lens"], s["lse"], s["out"], cu_tokens=s["cu"],
                                      earlier=s["earlier"], decay=case["decay"], workspace=ws, check_status=False)
        if op == "evict":
            smla.cache_free(cache, s["new_table"], workspace=ws, check_status=False)
            new = smla.cache_evict(cache, s["table"], s["lens"], s["weights"], case["keep"], first=case["first"],
                                   recent=case["recent"], workspace=ws, check_status=False,
                                   out=(s["new_table"], s["new_lens"], s["new_weights"], s["kept"]))
        else:
            s["refcount"].copy_(s["count0"])
            smla.cache_reorder(cache, s["table"], s["lens"], s["parents"], weights=s["weights"], workspace=ws,
                               check_status=False, out=(s["new_table"], s["new_lens"], s["new_weights"]))
    else:
        if op == "select":
            return _select_plain(s)
        if op == "watch":
            return _watch_plain(s)
        if op == "evict":
            new = _evict_plain(s)
        else:
            s["refcount"].copy_(s["count0"])
            _reorder_plain(s)
    values = s["codes"].view(torch.float8_e4m3fn)
    if op == "evict":
        return (*new, s["refcount"], values, s["scales"])
    return s["new_table"], s["new_lens"], s["new_weights"], s["refcount"], values, s["scales"]


# ----------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return _select_exact(case, s)
    page, block = case["page"], case["block"]
    table, codes, scales = s["table"].tolist(), s["codes"].view(torch.float8_e4m3fn), s["scales"].double()
    if case["op"] == "watch":
        out = s["out"].double()
        cu, seen = s["cu"].tolist(), s["lens"].tolist()
        for b in range(case["B"]):
            n = max(seen[cu[b]:cu[b + 1]])
            at = torch.arange(n, device="cuda")
            where = s["table"][b].long()[at // page]
            x = codes[where, at % page].double() * scales[where, at % page // block, None]
            total = case["decay"] * s["earlier"][b, :n].double()
            for t in range(cu[b], cu[b + 1]):
                logits = s["q"][t].double() @ x[: seen[t]].T / D ** 0.5
                total[: seen[t]] += torch.exp(logits - s["lse"][t].double()[:, None]).sum(0)
            out[b, :n] = total
        return out
    lens, count = s["lens"].tolist(), s["refcount"].tolist()
    values, new_scales = codes.to(torch.float64), scales.clone()
    rows, width = s["table"].shape
    new = [[-1] * width for _ in range(rows)]
    free = iter([i for i, c in enumerate(count) if c == 0])
    if case["op"] == "reorder":
        parents = s["parents"].tolist()
        heirs, spare = {}, []
        for i, p in enumerate(parents):
            heirs.setdefault(p, i)
        for p in range(rows):
            if p not in heirs:
                rest = table[p][lens[p] // page] if lens[p] % page else -1
                if rest >= 0 and count[rest] == 1:
                    spare.append(rest)
                for e in table[p]:
                    if e >= 0:
                        count[e] -= 1
        for i, p in enumerate(parents):
            if heirs[p] == i:
                new[i] = list(table[p])
                continue
            full, rest = divmod(lens[p], page)
            for j in range(full):
                new[i][j] = table[p][j]
                count[table[p][j]] += 1
            if rest:
                to = spare.pop(0) if spare else next(free)
                new[i][full], count[to] = to, 1
                values[to], new_scales[to] = values[table[p][full]], new_scales[table[p][full]]
        weights = None
        if s["weights"] is not None:
            weights = torch.zeros_like(s["weights"], dtype=torch.float64)
            for i, p in enumerate(parents):
                weights[i, : lens[p]] = s["weights"][p, : lens[p]].double()
        return (torch.tensor(new), torch.tensor([lens[p] for p in parents]), weights, torch.tensor(count), values,
                new_scales)
    keep = case["keep"]
    weights = torch.zeros_like(s["weights"], dtype=torch.float64)
    kept = torch.full((rows, keep), -1)
    for b in range(rows):
        n = lens[b]
        w = s["weights"][b, :n].double().cpu()
        w[: case["first"]] = math.inf
        w[max(0, n - case["recent"]):] = math.inf
        best = sorted(range(n), key=w.neg().tolist().__getitem__)[:keep]      # (sorted keeps the order of ties)
        best = torch.tensor(sorted(best))
        m = best.shape[0]
        kept[b, :m] = best
        best = best.cuda()
        weights[b, :m] = s["weights"][b, best].double()
        where = s["table"][b].long()[best // page]
        sc = scales[where, best % page // block]
        x = codes[where, best % page].double()
        for j in range(0, m, page):
            to = next(free)
            new[b][j // page], count[to] = to, 1
            for k in range(j, min(j + page, m), block):
                part = slice(k, min(k + block, j + page, m))
                size = sc[part].max()
                y = x[part] * (sc[part] / size)[:, None]
                # e4m3: 4 significant bits, spacing 2^-9 at the least
                gap = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                values[to, k - j: part.stop - j] = torch.round(y / gap) * gap
                new_scales[to, (k - j) // block] = size
    return (torch.tensor(new), torch.tensor([min(n, keep) for n in lens]), weights, kept, torch.tensor(count), values,
            new_scales)


def _select_exact(case, s):
    K, n, V = case["K"], case["n"], case["V"]
    parents, tokens, scores = [], [], []
    for b in range(case["B"]):
        found = []
        for k in range(K):
            x = s["logits"][b * K + k].double()
            before = float(s["scores"][b, k])
            if s["done"] is not None and bool(s["done"][b, k]):
                found.append((-before, k, s["eos"]))
                continue
            x = before + (x - torch.logsumexp(x, 0))
            least = torch.topk(x, min(n, V))[0][-1]
            at = torch.nonzero((x >= least) & torch.isfinite(x))[:, 0]
            found += [(-v, k, i) for v, i in zip(x[at].tolist(), at.tolist())]
        found = sorted(found)[:n]
        rest = n - len(found)
        parents.append([b * K + k for _, k, _ in found] + [-1] * rest)
        tokens.append([i for _, _, i in found] + [-1] * rest)
        scores.append([-v for v, _, _ in found] + [-math.inf] * rest)
    return torch.tensor(parents), torch.tensor(tokens), torch.tensor(scores, dtype=torch.float64)
