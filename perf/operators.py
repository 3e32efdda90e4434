"""Cases of the 8-bit paged key/value cache: what each operator computes in
elementary torch operations, and the library's calls beside it.

Cache of one layer: codes k [pages, heads, P, d] and v [pages, heads, P / 16,
d, 16] (the values of 16 tokens lie together, transposed) as int8 or e4m3,
with one fp32 scale per page (block of P tokens) and head.  A row of `table`
lists the pages of one sequence, `lens` its tokens; token t lies in slot t % P
of page table[t // P].

  store     the new keys and values of each sequence are quantised into its
            pages, and its last tokens are read back
  attend    softmax attention of each sequence's newest queries over its cache
  fork      finished sequences leave, others are forked into their rows: whole
            pages shared, the last part-filled page copied in every layer
  turnover  finished sequences leave, new ones take the lowest free pages
  compact   pages move down into the holes of the pool
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
TOP = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TINY = torch.finfo(torch.float32).tiny


def listed():
    return [
        # one decode step of the GPT-2 124M batch: 32 sequences between the 128-token prompt and 512 tokens
        dict(name="store-token", op="store", kind="int8", dtype="bf16", batch=32, kv=12, d=64, page=16, lo=128, hi=512, new=1),
        # prefill of a batch of prompts of a grouped-head model, ragged
        dict(name="store-prompts", op="store", kind="e4m3", dtype="fp16", batch=64, kv=8, d=128, page=64, lo=17, hi=2048, new=2048),
        # greedy decoding of one sequence at GPT-2 124M's head layout: latency
        dict(name="attend-one", op="attend", kind="int8", dtype="bf16", batch=1, kv=12, group=1, d=64, page=16, lo=512, hi=512, new=1),
        # the same model's batch of 32 between prompt and end
        dict(name="attend-batch", op="attend", kind="int8", dtype="bf16", batch=32, kv=12, group=1, d=64, page=16, lo=128, hi=512, new=1),
        # one very long document, grouped heads, an odd length
        dict(name="attend-long", op="attend", kind="e4m3", dtype="bf16", batch=1, kv=8, group=4, d=128, page=64, lo=131071, hi=131071, new=1),
        # a server's mixed batch: one to five new tokens each, contexts from a few tokens to 16K, empty sequences among them
        dict(name="attend-ragged", op="attend", kind="int8", dtype="fp16", batch=64, kv=8, group=4, d=64, page=32, lo=0, hi=16384, new=5),
        # one prompt split into beams, GPT-2 124M
        dict(name="fork-beams", op="fork", layers=12, kv=12, d=64, page=16, sources=1, ways=7, lo=137, hi=137),
        # many continuations of a few prompts at once
        dict(name="fork-many", op="fork", layers=12, kv=8, d=128, page=64, sources=4, ways=64, lo=300, hi=1000),
        # page bookkeeping of a batch of 32 with 1024-token rows
        dict(name="turnover-batch", op="turnover", rows=32, max_pages=64, page=16, pages=2048, gone=8),
        # the same of a large server
        dict(name="turnover-large", op="turnover", rows=1024, max_pages=512, page=16, pages=262144, gone=301),
        # the packed 8 x 512 model's pool with holes
        dict(name="compact-small", op="compact", layers=4, kv=6, d=32, page=16, rows=8, max_pages=32, pages=256, live=0.6),
        # a gigabyte of cache, a bit over half of it in use
        dict(name="compact-large", op="compact", layers=4, kv=8, d=128, page=32, rows=64, max_pages=64, pages=4097, live=0.55),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "store", "attend", "attend", "attend", "fork", "turnover", "compact"])
    kv, d, page = rng.choice([1, 2, 3, 4, 6, 8, 12]), rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
    if op in ("store", "attend"):
        batch = _log(rng, 1, 128)
        hi = max(1, min(131072, int((8 << 20) // (batch * kv)) if op == "store" else (1 << 20) // batch, int((1 << 27) // (batch * kv * d))))
        hi = _log(rng, 1, hi)
        c = dict(op=op, kind=rng.choice(["int8", "e4m3"]), dtype=rng.choice(["bf16", "fp16"]), batch=batch, kv=kv, d=d, page=page, lo=rng.choice([0, 1, hi, max(1, hi // 3)]), hi=hi)
        c["new"] = rng.choice([1, 1, 2, 5, hi, hi]) if op == "store" else rng.choice([1, 1, 1, 2, 5, 8])
        if op == "attend":
            c["group"] = rng.choice([1, 1, 2, 3, 4, 5, 8])
        return c
    if op == "fork":
        sources, layers = _log(rng, 1, 16), rng.randint(1, 12)
        ways = _log(rng, 1, max(1, min(256 // sources, (100 << 20) // (layers * kv * d * page * sources))))
        hi = _log(rng, 1, 40 * page)
        return dict(op=op, layers=layers, kv=kv, d=d, page=page, sources=sources, ways=ways, lo=max(1, hi // rng.randint(1, 3)), hi=hi)
    rows, max_pages = _log(rng, 1, 1024 if op == "turnover" else 64), _log(rng, 1, 256 if op == "turnover" else 64)
    pages = rows * max_pages + rng.randint(0, 100)
    if op == "turnover":
        return dict(op=op, rows=rows, max_pages=max_pages, page=page, pages=pages, gone=rng.randint(1, rows))
    layers = rng.randint(1, max(1, min(4, (128 << 20) // (pages * kv * d * page))))
    return dict(op=op, layers=layers, kv=kv, d=min(d, 64), page=min(page, 32), rows=rows, max_pages=max_pages, pages=pages, live=round(rng.uniform(0.2, 0.95), 3))


def _rng(case):
    # lengths belong to the case; the values in the tensors come from the seed
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _spread(rng, lo, hi, n):
    # contexts spread over their logarithm; the first one is the longest
    out = [int((lo + 1) * ((hi + 1) / (lo + 1)) ** rng.random()) - 1 for _ in range(n)]
    return [hi] + [min(hi, max(lo, x)) for x in out[1:]]


def _batch(case):
    """(tokens, new tokens) of every sequence."""
    r = _rng(case)
    lens = _spread(r, case["lo"], case["hi"], case["batch"])
    if case["op"] == "store":
        return lens, [min(n, case["new"]) for n in lens]
    return lens, [case["new"] if case["batch"] == 1 or case["new"] == 1 else r.randint(1, case["new"]) for _ in lens]


def _back(case, lens, new):
    # the tokens read back: the new ones, and what else of their pages an append may have rescaled
    return [min(n, max(m, case["page"])) for n, m in zip(lens, new)]


def _pages(n, page):
    return -(-n // page)


def work(case):
    op = case["op"]
    if op == "store":
        lens, new = _batch(case)
        e = case["kv"] * case["d"]
        touched = sum(_pages(n, case["page"]) - (n - m) // case["page"] for n, m in zip(lens, new) if m)
        # keys and values: in at 16 bits, out at 8; read back in at 8, out at 16; the scales of each touched page both ways
        return {"bytes": 2 * (sum(new) * e * 3 + sum(_back(case, lens, new)) * e * 3 + touched * case["kv"] * 8), "flops": 2 * 2 * sum(new) * e}
    if op == "attend":
        lens, new = _batch(case)
        e, h = case["kv"] * case["d"], case["kv"] * case["group"]
        pairs = sum(sum(max(0, n - i) for i in range(m)) for n, m in zip(lens, new))
        blocks = sum(_pages(n, case["page"]) for n in lens)
        return {"bytes": 2 * sum(lens) * e + 2 * 4 * blocks * case["kv"] + sum(new) * h * (4 * case["d"] + 4) + 4 * blocks, "flops": 4 * pairs * h * case["d"]}
    if op == "fork":
        s = _fork_lens(case)
        part = sum(case["ways"] for n in s if n % case["page"])
        per = 2 * case["layers"] * case["kv"] * (case["page"] * case["d"] + 4)
        shared = sum(_pages(n, case["page"]) for n in s) * case["ways"]
        return {"bytes": 2 * part * per + 4 * 4 * shared, "flops": shared}
    if op == "turnover":
        old, add = _turnover_lens(case)
        moved = sum(_pages(old[r], case["page"]) + _pages(a, case["page"]) for r, a in enumerate(add) if a)
        # every page's reference count is looked at once; a page that leaves or comes changes its count and its place in a row
        return {"bytes": 4 * case["pages"] + 12 * moved + 12 * case["rows"], "flops": case["pages"]}
    moves, entries = _compact_moves(case)
    return {"bytes": 2 * moves * (2 * case["layers"] * case["kv"] * (case["page"] * case["d"] + 4)) + 8 * entries + 4 * case["pages"], "flops": case["pages"]}


# ---- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _normal(g, *shape):
    # channels of unlike size, as keys have them
    x = torch.randn(*shape, generator=g, device="cuda")
    return x * torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))


def _codes(g, kind, pages, kv, page, d):
    """Random codes [pages, kv, page, d] with their scales [pages, kv]."""
    x = _normal(g, pages, kv, page, d)
    s = x.abs().amax((2, 3)) / TOP[kind]
    return _quantise(x, s, kind), s


def _lay_v(x):
    n, h, p, d = x.shape
    return x.view(torch.uint8).view(n, h, p // 16, 16, d).transpose(3, 4).contiguous()


def _table(g, counts, max_pages, pages):
    """Rows of page ids in random order, -1 behind each row's end."""
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[:sum(counts)]
    at = torch.arange(max_pages, device="cuda")[None, :] < _ints(counts)[:, None]
    t = torch.full((len(counts), max_pages), -1, dtype=torch.int32, device="cuda")
    t[at] = ids
    return t


def _starts(new):
    out = [0]
    out += [sum(new[:i + 1]) for i in range(len(new))]
    return _ints(out)


def _fork_lens(case):
    r = _rng(case)
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["sources"] - 1)]


def _turnover_lens(case):
    r = _rng(case)
    top = case["max_pages"] * case["page"]
    room = max(1, min(top, (case["pages"] * case["page"]) // (2 * case["rows"])))
    old = [r.randint(1, room) for _ in range(case["rows"])]
    gone = set(r.sample(range(case["rows"]), case["gone"]))
    return old, [r.randint(1, room) if i in gone else 0 for i in range(case["rows"])]


def _compact_lens(case):
    r = _rng(case)
    want = max(1, int(case["live"] * case["pages"] / case["rows"]))
    return [min(case["max_pages"], max(1, want + r.randint(-want // 2, want // 2))) * case["page"] - r.randint(0, case["page"] - 1) for _ in range(case["rows"])]


def _compact_moves(case):
    used = sum(_pages(n, case["page"]) for n in _compact_lens(case))
    # pages lie at random places: of `used` live ones, those above the first `used` places move
    return int(used * (1 - used / case["pages"])), used


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("store", "attend"):
        lens, new = _batch(case)
        page, kv, d, kind = case["page"], case["kv"], case["d"], case["kind"]
        counts = [_pages(n, page) for n in lens]
        pages = sum(counts) + 3
        s = {"case": dict(case), "lens": _ints(lens), "start": None if new == [1] * len(new) else _starts(new), "rows": sum(new)}
        s["table"] = _table(g, counts, max(1, max(counts)), pages)
        s["k"], s["k_scale"] = _codes(g, kind, pages, kv, page, d)
        v, s["v_scale"] = _codes(g, kind, pages, kv, page, d)
        s["v"] = _lay_v(v).view(CODE[kind])[None]
        s["k"], s["k_scale"], s["v_scale"] = s["k"][None], s["k_scale"][None], s["v_scale"][None]
        if op == "attend":
            s["q"] = (1.5 * torch.randn(sum(new), kv * case["group"], d, generator=g, device="cuda")).to(DT[case["dtype"]])
            return s
        s["new_k"] = _normal(g, sum(new), kv, d).to(DT[case["dtype"]])
        s["new_v"] = _normal(g, sum(new), kv, d).to(DT[case["dtype"]])
        back = _back(case, lens, new)
        s["back"], s["back_rows"] = _starts(back), sum(back)
        return s
    if op == "fork":
        src = _fork_lens(case)
        n, page = case["sources"] * case["ways"], case["page"]
        # rows: the sources, then the rows of finished sequences that the forks take over
        r = _rng(case)
        lens = src + [r.randint(1, 2 * page) for _ in range(n)]
        table = _table(g, [_pages(x, page) for x in lens], max(_pages(max(lens), page), 2), sum(_pages(x, page) for x in lens) + n)
        s = {"table": table, "src": _ints([i % case["sources"] for i in range(n)]), "dst": _ints([case["sources"] + i for i in range(n)])}
        s["n_pages"] = sum(_pages(x, page) for x in lens) + n
    elif op == "turnover":
        old, add = _turnover_lens(case)
        lens, page = old, case["page"]
        s = {"table": _table(g, [_pages(x, page) for x in old], case["max_pages"], case["pages"]), "n_pages": case["pages"]}
        s["add"], s["gone"] = _ints(add), _ints([i for i, a in enumerate(add) if a])
    else:
        lens, page = _compact_lens(case), case["page"]
        s = {"table": _table(g, [_pages(x, page) for x in lens], case["max_pages"], case["pages"]), "n_pages": case["pages"]}
    s["lens"], s["case"] = _ints(lens), dict(case)
    s["ref"] = torch.zeros(s["n_pages"], dtype=torch.int32, device="cuda")
    s["ref"][s["table"][s["table"] >= 0].long()] = 1
    if op == "compact":
        s["table0"], s["ref0"] = s["table"].clone(), s["ref"].clone()
    layers, kv, d = case.get("layers", 1), case.get("kv", 1), case.get("d", 16)
    shape = (layers, s["n_pages"], kv) if op != "turnover" else (1, 1, 1)   # bookkeeping alone touches no codes
    fill = lambda *n: torch.randint(0, 120, n, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    s["k"], s["v"] = fill(*shape, page, d), fill(*shape, page // 16, d, 16)
    s["k_scale"], s["v_scale"] = (torch.rand(shape, generator=g, device="cuda") + 0.5 for _ in range(2))
    return s


# ---- plain forms

def _quantise(x, s, kind):
    s = s[..., None, None] if s.dim() < x.dim() else s
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    y = (x * inv).clamp(-TOP[kind], TOP[kind])
    return (torch.round(y) if kind == "int8" else y).to(CODE[kind])


def _rows(start, rows, lens):
    """(sequence, position) of each row: the last row of a sequence is its newest token."""
    r = torch.arange(rows, device="cuda")
    if start is None:
        return r, lens.long() - 1
    b = torch.searchsorted(start[1:].contiguous(), r.to(torch.int32), right=True)
    return b, lens.long()[b] - (start.long()[b + 1] - r)


def _at(s, b, pos, page):
    return s["table"][b, pos // page].long(), pos % page


def _store(s):
    c = s["case"]
    page, kind, kv, d = c["page"], c["kind"], c["kv"], c["d"]
    b, pos = _rows(s["start"], s["rows"], s["lens"])
    pid, slot = _at(s, b, pos, page)
    pages, job = torch.unique(pid, return_inverse=True)
    n = pages.numel()
    first = torch.full((n,), page, device="cuda").scatter_reduce(0, job, slot, "amin")
    kept = torch.arange(page, device="cuda")[None, :] < first[:, None]
    for x, codes, scales, is_v in ((s["new_k"], s["k"], s["k_scale"], False), (s["new_v"], s["v"], s["v_scale"], True)):
        dense = torch.zeros(n, kv, page, d, device="cuda")
        dense[job, :, slot] = x.float()
        fresh = dense.abs().amax((2, 3)) / TOP[kind]
        before = torch.where(first[:, None] > 0, scales[0, pages], torch.zeros_like(fresh))
        after = torch.maximum(before, torch.where(fresh < TINY, torch.zeros_like(fresh), fresh))
        held = codes[0].view(torch.uint8)[pages]
        if is_v:
            held = held.transpose(3, 4).reshape(n, kv, page, d)
        held = held.contiguous().view(CODE[kind])
        ratio = torch.where(after > 0, before / after, torch.zeros_like(after))[..., None, None]
        moved = held.float() * ratio
        moved = (torch.round(moved) if kind == "int8" else moved).to(CODE[kind])
        put = torch.where(kept[:, None, :, None], torch.where(ratio == 1, held.view(torch.uint8), moved.view(torch.uint8)), _quantise(dense, after, kind).view(torch.uint8))
        codes[0].view(torch.uint8)[pages] = _lay_v(put) if is_v else put
        scales[0, pages] = after
    b, pos = _rows(s["back"], s["back_rows"], s["lens"])
    k, v = _read(s, b, pos)
    return {"k": k.to(DT[c["dtype"]]), "v": v.to(DT[c["dtype"]]), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _read(s, b, pos):
    """The values in 32 bits that the cache holds of the tokens `pos` of sequences `b`: [..., heads, d] each."""
    kind = s["case"]["kind"]
    pid, slot = _at(s, b, pos, s["case"]["page"])
    k = s["k"][0].view(torch.uint8)[pid, :, slot].view(CODE[kind]).float() * s["k_scale"][0, pid][..., None]
    v = s["v"][0].view(torch.uint8)[pid, :, slot // 16, :, slot % 16].view(CODE[kind]).float() * s["v_scale"][0, pid][..., None]
    return k, v


def _attend(s):
    c = s["case"]
    kv, group, d, most, top = c["kv"], c["group"], c["d"], c["new"], c["hi"]
    B = s["lens"].numel()
    b, pos = _rows(s["start"], s["rows"], s["lens"])
    if s["rows"] == 0 or top == 0:
        return {"out": torch.zeros_like(s["q"]), "lse": torch.full((s["rows"], kv * group), -math.inf, device="cuda")}
    at = (s["lens"].long()[b] - 1 - pos)       # 0: the newest query of its sequence
    q = torch.zeros(B, most, kv * group, d, device="cuda")
    q[b, at] = s["q"].float()
    t = torch.arange(top, device="cuda")
    inside = t[None, :] < s["lens"][:, None]
    k, v = _read(s, torch.arange(B, device="cuda")[:, None].expand(B, top), torch.where(inside, t[None, :], torch.zeros_like(t)[None, :]))
    q = q.view(B, most, kv, group, d).permute(0, 2, 1, 3, 4).reshape(B, kv, most * group, d)
    x = (q @ k.permute(0, 2, 3, 1)) * (d ** -0.5)
    limit = s["lens"].long()[:, None] - torch.arange(most, device="cuda")[None, :]    # tokens that a query may see
    seen = (t[None, None, :] < limit[:, :, None])[:, None, :, None, :].expand(B, kv, most, group, top).reshape(B, kv, most * group, top)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    w = torch.exp(x - m)
    total = w.sum(-1, keepdim=True)
    out = (w @ v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + m)[..., 0]
    out = out.view(B, kv, most, group, d).permute(0, 2, 1, 3, 4).reshape(B, most, kv * group, d)
    lse = lse.view(B, kv, most, group).permute(0, 2, 1, 3).reshape(B, most, kv * group)
    return {"out": out[b, at].to(s["q"].dtype), "lse": lse[b, at].contiguous()}


def _drop(s, rows):
    """The sequences in `rows` leave: their references go, their rows empty."""
    ids = s["table"][rows.long()]
    hold = ids >= 0
    s["ref"].index_add_(0, ids.clamp(min=0).long().view(-1), -hold.to(torch.int32).view(-1))
    s["table"][rows.long()] = -1
    s["lens"][rows.long()] = 0


def _fork(s):
    page = s["case"]["page"]
    _drop(s, s["dst"])
    src, dst = s["src"].long(), s["dst"].long()
    n = s["lens"][src].long()
    count, part = (n + page - 1) // page, n % page > 0
    free = torch.nonzero(s["ref"] == 0)[:, 0]
    ids = s["table"][src].clone()
    last = (count - 1)[:, None]
    fresh = free[torch.cumsum(part, 0) - part.long()].to(torch.int32)     # the i-th pair in need of a page takes the i-th lowest free one
    old = ids.gather(1, last)[:, 0]
    ids.scatter_(1, last, torch.where(part, fresh, old)[:, None])
    s["table"][dst] = ids
    s["lens"][dst] = s["lens"][src]
    s["ref"].index_add_(0, ids.clamp(min=0).long().view(-1), (ids >= 0).to(torch.int32).view(-1))
    a, z = old[part].long(), fresh[part].long()
    for t in (s["k"], s["v"]):
        u = t.view(torch.uint8)
        u[:, z] = u[:, a]
    for t in (s["k_scale"], s["v_scale"]):
        t[:, z] = t[:, a]
    return {"done": torch.ones_like(s["dst"]), "table": s["table"], "lens": s["lens"], "ref": s["ref"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _turnover(s):
    page = s["case"]["page"]
    _drop(s, s["gone"])
    have = (s["lens"].long() + page - 1) // page
    want = (s["lens"].long() + s["add"].long() + page - 1) // page
    p = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    need = (p >= have[:, None]) & (p < want[:, None])
    free = torch.nonzero(s["ref"] == 0)[:, 0].to(torch.int32)
    ids = free[:int(need.sum())]
    s["table"][need] = ids
    s["ref"][ids.long()] = 1
    s["lens"] += s["add"]
    return {"table": s["table"], "lens": s["lens"], "ref": s["ref"]}


def _compact(s):
    live = s["ref"] > 0
    n = int(live.sum())
    z = torch.nonzero(~live[:n])[:, 0]
    a = torch.nonzero(live[n:])[:, 0] + n
    to = torch.arange(live.numel(), device="cuda", dtype=torch.int32)
    to[a] = z.to(torch.int32)
    for t in (s["k"], s["v"]):
        u = t.view(torch.uint8)
        u[:, z] = u[:, a]
    for t in (s["k_scale"], s["v_scale"]):
        t[:, z] = t[:, a]
    s["ref"][z] = s["ref"][a]
    s["ref"][a] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], s["table"]))
    return {"table": s["table"], "ref": s["ref"], "n_live": n, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ---- the library's calls

def _handle(s):
    if "cache" not in s:
        from scratch_decoder_only_b200.kv8 import KV8Batch, KV8Cache, KV8Pool
        if s["case"]["op"] == "turnover":
            s["cache"] = KV8Pool(s["table"], s["lens"], s["ref"], s["case"]["page"])
            return s["cache"]
        s["cache"] = KV8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["lens"], s.get("ref"))
        if "rows" in s:
            s["batch"] = KV8Batch(s["table"], s["lens"], s["start"], s["rows"])
        if "back" in s:
            s["reading"] = KV8Batch(s["table"], s["lens"], s["back"], s["back_rows"])
    return s["cache"]


def _own(s):
    c, op = _handle(s), s["case"]["op"]
    if op == "store":
        c.append(0, s["new_k"], s["new_v"], s["batch"])
        k, v = c.read(0, s["reading"], DT[s["case"]["dtype"]])
        return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "attend":
        out, lse = c.attention(0, s["q"], s["batch"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "fork":
        c.free(s["dst"])
        done = c.fork(s["src"], s["dst"])
        return {"done": done, "table": s["table"], "lens": s["lens"], "ref": s["ref"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "turnover":
        c.free(s["gone"])
        c.extend(s["add"])
        return {"table": s["table"], "lens": s["lens"], "ref": s["ref"]}
    n = c.compact()
    return {"table": s["table"], "ref": s["ref"], "n_live": n, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    if state["case"]["op"] == "compact":
        # the same holes for every pass; the codes need no setting back, for a move leaves its source as it was
        state["table"].copy_(state["table0"])
        state["ref"].copy_(state["ref0"])
    if own:
        return _own(state)
    return {"store": _store, "attend": _attend, "fork": _fork, "turnover": _turnover, "compact": _compact}[state["case"]["op"]](state)


# ---- 64-bit values, one sequence at a time

def _grid(y, kind):
    """`y` in 64 bits on the grid of the code type, half to even."""
    if kind == "int8":
        return torch.round(y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _held(layer_codes, scales, is_v):
    x = layer_codes.double() if not is_v else layer_codes.double().transpose(-1, -2).flatten(2, 3)
    return (x * scales.double()[:, :, None, None]).transpose(1, 2).flatten(0, 1)


def _tokens(s, which, ids):
    """Tokens [n * P, heads, d] in 64 bits of the pages `ids`."""
    u = s[which][0].view(torch.uint8)[ids].view(s[which].dtype)
    return _held(u, s[which + "_scale"][0][ids], which == "v")


def exact(case, seed):
    if case["op"] not in ("store", "attend"):
        return None
    s = prepare(case, seed)
    lens, new = _batch(case)
    page, kv, d = case["page"], case["kv"], case["d"]
    outs = {"k": [], "v": []} if case["op"] == "store" else {"out": [], "lse": []}
    scales = {w: s[w + "_scale"].double().clone() for w in ("k", "v")}
    at = 0
    for b, (n, m, back) in enumerate(zip(lens, new, _back(case, lens, new))):
        ids = s["table"][b, :_pages(n, page)].long()
        if case["op"] == "attend":
            q = s["q"][at:at + m].double().view(m, kv, case["group"], d)
            x = torch.einsum("ihgd,thd->ihgt", q, _tokens(s, "k", ids)[:n]) / math.sqrt(d)
            hidden = torch.arange(n, device="cuda")[None, :] > torch.arange(n - m, n, device="cuda")[:, None]
            x = x.masked_fill(hidden[:, None, None, :], -math.inf)
            some = (~hidden).any(-1)[:, None, None, None]
            p = torch.softmax(x, -1) if n else x
            outs["out"].append(torch.where(some, torch.einsum("ihgt,thd->ihgd", p.nan_to_num(0.0), _tokens(s, "v", ids)[:n]), 0.0).reshape(m, kv * case["group"], d))
            outs["lse"].append(torch.logsumexp(x, -1).reshape(m, -1) if n else torch.full((m, kv * case["group"]), -math.inf, dtype=torch.float64, device="cuda"))
        else:
            f, kind = (n - m) // page, case["kind"]      # the first page that the new tokens enter
            inside = (n - m) % page
            for w in ("k", "v"):
                ids_f = ids[f:]
                was = scales[w][0][ids_f]
                x = torch.zeros(ids_f.numel() * page, kv, d, dtype=torch.float64, device="cuda")
                x[inside:inside + m] = s["new_" + w][at:at + m].double()
                a = x.view(-1, page, kv, d).abs().amax((1, 3)) / TOP[kind]
                if not inside:
                    was = torch.zeros_like(was)
                was = torch.cat([was[:1], torch.zeros_like(was[1:])])
                now = torch.maximum(a, was)
                each = now.repeat_interleave(page, 0)[..., None].clamp(min=1e-300)
                y = _grid(x / each, kind) * each
                if inside:
                    old = _tokens(s, w, ids_f[:1])[:inside]
                    up = (now[0] / was[0].clamp(min=1e-300))[None, :, None]
                    y[:inside] = torch.where(up > 1, _grid(old / each[:1], kind) * each[:1], old)
                scales[w][0][ids_f] = now
                before = _tokens(s, w, ids[:f])
                outs[w].append(torch.cat([before, y])[n - back:n])
        at += m
    got = {name: torch.cat(v) for name, v in outs.items()}
    if case["op"] == "store":
        got |= {"k_scale": scales["k"], "v_scale": scales["v"]}
    return got
