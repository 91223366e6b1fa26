"""Measured cases of the operators for many answers to one prompt: the pages of
the 8-bit key/value cache (growing, forking, freeing, compacting, copying), the
attention of sequences that share a prefix, and log probabilities of given
tokens with entropy and top alternatives, with their gradient.

`own` false: the plain form, elementary torch operations in fp32.  `own` true:
the calls that a user of ternary_weight_absmean_amd makes.  `exact` evaluates
the definitions in 64 bits.  Sequence lengths and parents are functions of the
case alone (the work of a case does not depend on the seed); values and the
places of pages come from the seed.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
BF16 = torch.bfloat16


# ---- cases ----

def listed():
    fork = {"op": "fork"}
    compact = {"op": "compact"}
    shared = {"op": "shared"}
    score = {"op": "logprobs"}
    train = {"op": "train"}
    return [
        # a beam step: four beams of one short conversation pick their parents, 2B-shaped cache of a few blocks
        dict(fork, name="pages, four beams", seqs=4, children=4, ctx=700, prompt=500, width=4, consume=True, new=1, heads=5,
             dim=128, page=64, layers=4, spare=300),
        # 24 prompts fork into 8 answers each and stay (they may be asked again), 70B-shaped cache of a few blocks
        dict(fork, name="pages, answers", seqs=24, children=192, ctx=3000, prompt=0, width=1, consume=False, new=5, heads=8,
             dim=128, page=64, layers=4, spare=2000),
        # two of nine short sequences have ended, small pages
        dict(compact, name="compact, few", seqs=9, ctx=300, ended=2, heads=2, dim=64, page=16, layers=3, spare=20),
        # half of a batch has ended, the pool is scattered, 70B-shaped
        dict(compact, name="compact, half", seqs=64, ctx=1500, ended=32, heads=8, dim=128, page=64, layers=4, spare=500),
        # four answers to one prompt, one token each
        dict(shared, name="shared, four answers", groups=1, width=4, prefix=1000, ctx=60, new=1, hq=20, hkv=5, dim=128, page=64),
        # a decode batch of answers to two long prompts
        dict(shared, name="shared, decode batch", groups=2, width=32, prefix=16384, ctx=500, new=1, hq=64, hkv=8, dim=128,
             page=64),
        # questions of several users behind one long instruction, read for the first time
        dict(shared, name="shared, prompts", groups=1, width=6, prefix=12000, ctx=0, new=409, hq=20, hkv=5, dim=128, page=32),
        # one decoded token with 20 alternatives, a temperature
        dict(score, name="logprobs, one token", m=1, n=128256, bf16=True, top=20, scale=1.4, masked=0.0),
        # a decode batch whose answers may use part of the vocabulary only
        dict(score, name="logprobs, decode batch", m=64, n=128256, bf16=True, top=20, scale=1.0, masked=0.5),
        # the tokens of given answers scored, fp32 logits with rows of odd length
        dict(score, name="logprobs, given answers", m=333, n=50001, bf16=False, top=5, scale=1.0, masked=0.0),
        # a small training batch, fp32, odd rows
        dict(train, name="train, ragged", m=37, n=32003, bf16=False, scale=1.0, masked=0.0),
        # a training batch with the large vocabulary
        dict(train, name="train, batch", m=4096, n=128256, bf16=True, scale=1.0, masked=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fork", "compact", "shared", "shared", "logprobs", "train"])
    heads, dim = rng.randint(1, 8), rng.choice([64, 128, 16 * rng.randint(2, 16)])
    page = rng.choice([16, 32, 64, 128])
    if op == "fork":
        width = rng.choice([1, 2, 4])
        seqs = width * _log(rng, 1, 16)
        return {"op": op, "seqs": seqs, "children": rng.choice([seqs, _log(rng, 1, 192)]), "ctx": _log(rng, 2, 3000),
                "prompt": rng.choice([0, 200]), "width": width, "consume": rng.random() < 0.5, "new": rng.choice([1, rng.randint(2, 70)]),
                "heads": heads, "dim": dim, "page": page, "layers": rng.randint(1, 4), "spare": _log(rng, 10, 2000)}
    if op == "compact":
        seqs = _log(rng, 2, 64)
        return {"op": op, "seqs": seqs, "ctx": _log(rng, 2, 1500), "ended": rng.randint(0, seqs), "heads": heads, "dim": dim,
                "page": page, "layers": rng.randint(1, 4), "spare": _log(rng, 1, 500)}
    if op == "shared":
        hq = heads * rng.choice([1, 2, 4, 5, 8])
        groups, width = rng.randint(1, 4), _log(rng, 1, 32)
        if rng.random() < 0.6:  # decode: one token, or a few (a draft being verified)
            new, ctx = rng.choice([1, 1, rng.randint(2, 6)]), _log(rng, 1, 1000)
        else:
            new, ctx = _log(rng, 7, max(8, 1600 // (groups * width))), rng.choice([0, _log(rng, 1, 300)])
        most = 409 * 6 * 20 * 128 * 12000 // (groups * width * new * hq * dim)
        return {"op": op, "groups": groups, "width": width, "prefix": _log(rng, 16, max(17, min(16384, most))), "ctx": ctx, "new": new, "hq": hq,
                "hkv": heads, "dim": dim, "page": page}
    n = _log(rng, 100, 200000)
    case = {"op": op, "m": _log(rng, 1, min(4096, (1 << 28) // n)), "n": n, "bf16": rng.random() < 0.5,
            "scale": rng.choice([1.0, 0.5, 1.4]), "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20, rng.randint(2, 64)])
        case["m"] = _log(rng, 1, min(512, (1 << 25) // n))
    return case


_GOLDEN = 0.6180339887498949


def _spread(n):
    return [1.0 if s == 0 else 0.05 + 0.95 * ((s * _GOLDEN) % 1.0) for s in range(n)]


def _lengths(c):
    """Tokens that each sequence holds; rows of a prompt (`width` of them) have at least the prompt."""
    return [max(c.get("prompt", 0), int(c["ctx"] * f)) for f in _spread(c["seqs"])]


def _parents(c):
    """Children in order of beams that did well: some parents have several, some none."""
    n, k = c["seqs"], c["children"]
    if not c["consume"]:
        return [i * n // k for i in range(k)]
    return [int(n * ((i * _GOLDEN) % 1.0) ** 2) for i in range(k)]


def _kept(c):
    """Tokens that each sequence keeps: those that ended keep none."""
    order = sorted(range(c["seqs"]), key=lambda s: (s * _GOLDEN) % 1.0)
    gone = set(order[:c["ended"]])
    return [0 if s in gone else a for s, a in enumerate(_lengths(c))]


def _answers(c):
    """(tokens that each group shares, further tokens of each sequence, its new tokens)."""
    page, seqs = c["page"], c["groups"] * c["width"]
    prefix = [max(1, int(c["prefix"] * f) // page) * page for f in _spread(c["groups"])]
    return prefix, [int(c["ctx"] * f) for f in _spread(seqs)], [max(1, int(c["new"] * f)) for f in reversed(_spread(seqs))]


def work(c):
    op = c["op"]
    if op == "fork":
        page, length, parent = c["page"], _lengths(c), _parents(c)
        row = 2 * c["heads"] * c["dim"] * c["layers"]  # bytes of a token's codes
        seen, tokens, entries = set(), 0, 0
        for p in parent:
            if length[p] % page and (not c["consume"] or p in seen):
                tokens += length[p] % page
            seen.add(p)
            entries += -(-length[p] // page)
        return {"bytes": 2 * tokens * row + 16 * entries, "flops": entries}
    if op == "compact":
        pages = sum(-(-a // c["page"]) for a in _lengths(c))
        left = sum(-(-a // c["page"]) for a in _kept(c))
        all_pages = pages + c["spare"]
        moved = left * (all_pages - left) // all_pages  # as many as a scattered pool has above `left`, on average
        return {"bytes": 2 * moved * 2 * c["heads"] * c["page"] * c["dim"] * c["layers"] + 8 * all_pages + 8 * pages,
                "flops": all_pages}
    if op == "shared":
        prefix, ctx, new = _answers(c)
        width = c["width"]
        seen = sum(prefix) + sum(ctx) + sum(new)
        pairs = sum(n * (prefix[s // width] + a) + n * (n + 1) // 2 for s, (a, n) in enumerate(zip(ctx, new)))
        return {"bytes": 2 * seen * c["hkv"] * c["dim"] + 4 * sum(new) * c["hq"] * c["dim"],
                "flops": 4 * pairs * c["hq"] * c["dim"]}
    n = c["m"] * c["n"]
    size = 2 if c["bf16"] else 4
    if op == "logprobs":
        return {"bytes": n * size + c["m"] * (12 + 8 * c["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * size + 24 * c["m"], "flops": 14 * n}


# ---- inputs ----

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _caches(c, g, pages, heads, layers):
    """Caches of several blocks as earlier steps left them, pages that nobody holds with old data."""
    out = []
    for _ in range(layers):
        k, v = (torch.randint(-127, 128, (pages, heads, c["page"], c["dim"]), generator=g, device=DEV, dtype=torch.int8)
                for _ in range(2))
        ka, va = (0.5 + 4.0 * torch.rand(pages, heads, generator=g, device=DEV) for _ in range(2))
        out.append((k, v, ka, va))
    return out


def _quantised(x):
    """Codes and absmax of [..., tokens, dim] blocks."""
    a = x.abs().amax(dim=(-2, -1))
    return torch.round(x * (127.0 / a)[..., None, None]).to(torch.int8), a


def _heads(g, *shape):
    """Projections as they come out of a layer: normal, with a few strong channels."""
    x = torch.randn(*shape, generator=g, device=DEV)
    gain = torch.ones(shape[-1], device=DEV)
    gain[torch.randint(shape[-1], (4,), generator=g, device=DEV)] = 3.0
    return x * gain


def _logits(c, g):
    """Rows as a vocabulary's product gives them: normal, with some tokens that stand out, others forbidden."""
    m, n = c["m"], c["n"]
    x = torch.empty(m, n, dtype=BF16 if c["bf16"] else torch.float32, device=DEV)
    rows = max(1, (1 << 27) // n)
    for lo in range(0, m, rows):
        part = 2.0 * torch.randn(min(m, lo + rows) - lo, n, generator=g, device=DEV)
        if c["masked"]:
            part.masked_fill_(torch.rand(part.shape, generator=g, device=DEV) < c["masked"], -math.inf)
        likely = torch.randint(n, (part.shape[0], 8), generator=g, device=DEV)
        part.scatter_(1, likely, 3.0 + 3.0 * torch.randn(likely.shape, generator=g, device=DEV))
        x[lo:lo + rows] = part
    target = torch.randint(n, (m,), generator=g, device=DEV, dtype=torch.int32)
    best = torch.rand(m, generator=g, device=DEV) < 0.7  # most given tokens are likely ones
    target = torch.where(best, x.argmax(dim=1).int(), target)
    if m > 8:
        target[torch.arange(5, m, 8, device=DEV)] = -1  # tokens of a prompt: not scored
    return x, target


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"case": c}
    if op in ("fork", "compact"):
        page, length = c["page"], _lengths(c)
        stride = -(-(max(length) + c.get("new", 0)) // page)
        rows, used = [], 0
        for s, a in enumerate(length):
            have = -(-a // page)
            share = c.get("prompt", 0) // page if s % c.get("width", 1) else 0  # pages taken over from the prompt's first row
            rows.append((rows[s - s % c["width"]][:share] if share else []) + list(range(used, used + have - share)))
            used += have - share
        if op == "fork":
            extra = c["children"] * (1 + -(-c["new"] // page) + 1) + c["spare"]
        else:
            extra = c["spare"]
        pages = used + extra
        place = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
        table = torch.full((c["seqs"], stride), -1, dtype=torch.int32)
        refs = torch.zeros(pages, dtype=torch.int32)
        for s, r in enumerate(rows):
            table[s, :len(r)] = torch.tensor([place[i] for i in r], dtype=torch.int32)
            for i in r:
                refs[place[i]] += 1
        st["table0"], st["refs0"], st["length"] = table.to(DEV), refs.to(DEV), _ints(length)
        st["table"], st["refs"] = st["table0"].clone(), st["refs0"].clone()
        st["caches"] = _caches(c, g, pages, c["heads"], c["layers"])
        if op == "fork":
            st["parent"] = _ints(_parents(c))
            st["offsets"] = torch.arange(c["children"] + 1, dtype=torch.int32, device=DEV) * c["new"]
            st["max_len"] = max(length) + c["new"]
        else:
            st["keep"] = _ints(_kept(c))
            st["moves"] = pages // 2
    elif op == "shared":
        prefix, ctx, new = _answers(c)
        page, heads, width = c["page"], c["hkv"], c["width"]
        start = [prefix[s // width] + a for s, a in enumerate(ctx)]
        need = [-(-(a + n) // page) for a, n in zip(start, new)]
        rows, used = [], 0
        for s, n in enumerate(need):
            share = prefix[s // width] // page if s % width else 0
            rows.append((rows[s - s % width][:share] if share else []) + list(range(used, used + n - share)))
            used += n - share
        pages = used + 3
        place = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
        table = torch.zeros(len(need), max(need), dtype=torch.int32)
        for s, r in enumerate(rows):
            table[s, :len(r)] = torch.tensor([place[i] for i in r], dtype=torch.int32)
        st["table"] = table.to(DEV)
        st["kc"] = torch.empty(pages, heads, page, c["dim"], dtype=torch.int8, device=DEV)
        st["vc"], st["ka"] = torch.empty_like(st["kc"]), torch.empty(pages, heads, device=DEV)
        st["va"] = torch.empty_like(st["ka"])
        for lo in range(0, pages, 256):
            n = min(pages, lo + 256) - lo
            st["kc"][lo:lo + n], st["ka"][lo:lo + n] = _quantised(_heads(g, n, heads, page, c["dim"]))
            st["vc"][lo:lo + n], st["va"][lo:lo + n] = _quantised(torch.randn(n, heads, page, c["dim"], generator=g, device=DEV))
        st["total"], st["max_new"], st["max_len"] = sum(new), max(new), max(a + n for a, n in zip(start, new))
        st["start"], st["offsets"] = _ints(start), _ints([sum(new[:i]) for i in range(len(new) + 1)])
        st["group"], st["prefix"] = _ints([i * width for i in range(c["groups"] + 1)]), _ints(prefix)
        st["q"] = _heads(g, st["total"], c["hq"], c["dim"]).to(BF16)
    else:
        st["x"], st["target"] = _logits(c, g)
        if op == "train":
            m = c["m"]
            st["gl"] = torch.randn(m, generator=g, device=DEV) / m  # advantages
            st["gh"] = torch.full((m,), -0.01 / m, device=DEV)
            st["gz"] = 1e-4 * torch.rand(m, generator=g, device=DEV) / m
    if own:
        _handles(st, c)
    return st


def _handles(st, c):
    """What a program of the framework keeps from step to step: pool, cache and batch handles, output buffers."""
    import ternary_weight_absmean_amd as bl

    op = c["op"]
    st["bl"] = bl
    if op in ("fork", "compact"):
        st["pool"] = bl.KVPool(st["refs"], c["page"])
        st["kv"] = bl.KVCaches([bl.KVCache(*t) for t in st["caches"]])
        if op == "fork":
            n, stride = c["children"], st["table"].shape[1]
            st["out"] = dict(table=torch.empty(n, stride, dtype=torch.int32, device=DEV),
                             out_length=torch.empty(n, dtype=torch.int32, device=DEV),
                             copies=torch.empty(n, 3, dtype=torch.int32, device=DEV))
            st["short"] = torch.zeros(1, dtype=torch.int32, device=DEV)
            st["batch"] = bl.KVBatch(st["out"]["table"], st["out"]["out_length"], st["offsets"], n * c["new"], c["new"],
                                     st["max_len"])
        else:
            st["copies"] = torch.empty(st["moves"], 3, dtype=torch.int32, device=DEV)
            st["moved"] = torch.empty(1, dtype=torch.int32, device=DEV)
            st["workspace"] = torch.empty(bl.bl_kv_compact_workspace_bytes(st["pool"], st["moves"]), dtype=torch.uint8, device=DEV)
    elif op == "shared":
        st["cache"] = bl.KVCache(st["kc"], st["vc"], st["ka"], st["va"])
        st["batch"] = bl.KVBatch(st["table"], st["start"], st["offsets"], st["total"], st["max_new"], st["max_len"])
        st["shared"] = bl.KVShared(st["group"], st["prefix"], c["width"], max(_answers(c)[0]))
        st["out"] = torch.empty(st["total"], c["hq"], c["dim"], dtype=BF16, device=DEV)
        nbytes = bl.bl_attention_shared_workspace_bytes(st["cache"], st["batch"], st["shared"], c["hq"])
        st["workspace"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)
    else:
        m, t = c["m"], c.get("top", 0)
        st["out"] = {name: torch.empty(m, device=DEV) for name in ("logprob", "lse", "entropy")}
        if t:
            st["out"].update(top_id=torch.empty(m, t, dtype=torch.int32, device=DEV), top_logprob=torch.empty(m, t, device=DEV))
        nbytes = bl.bl_logprobs_workspace_bytes(m, c["n"], st["x"].dtype, t)
        st["workspace"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)
        if op == "train":
            st["dx"] = torch.empty_like(st["x"])


# ---- one pass ----

def run(st):
    op = st["case"]["op"]
    return (_OWN if own else _PLAIN)[op](st, st["case"])


def _own_fork(st, c):
    bl, pool, o = st["bl"], st["pool"], st["out"]
    st["refs"].copy_(st["refs0"])  # the pool as the step before left it
    st["short"].zero_()
    bl.bl_kv_fork(pool, st["table"], st["length"], st["parent"], keep_parents=not c["consume"], shortage=st["short"], **o)
    bl.bl_kv_copy(st["kv"], o["copies"])
    bl.bl_kv_grow(pool, st["batch"], shortage=st["short"])
    return [st["refs"], o["table"], o["out_length"], o["copies"], st["short"]] + [t for cache in st["caches"] for t in cache]


def _own_compact(st, c):
    bl, pool = st["bl"], st["pool"]
    st["refs"].copy_(st["refs0"])
    st["table"].copy_(st["table0"])
    bl.bl_kv_free(pool, st["table"], keep=st["keep"])
    bl.bl_kv_compact(pool, st["table"], st["moves"], copies=st["copies"], moved=st["moved"], workspace=st["workspace"])
    bl.bl_kv_copy(st["kv"], st["copies"], count=st["moved"])
    return [st["refs"], st["table"], st["copies"], st["moved"]] + [t for cache in st["caches"] for t in cache]


def _own_shared(st, c):
    return st["bl"].bl_attention_shared(st["cache"], st["batch"], st["shared"], st["q"], out=st["out"],
                                        workspace=st["workspace"])


def _own_logprobs(st, c):
    out = st["bl"].bl_logprobs(st["x"], st["target"], scale=c["scale"], top=c["top"], workspace=st["workspace"], **st["out"])
    return list(out if c["top"] else out[:3])


def _own_train(st, c):
    bl, o = st["bl"], st["out"]
    bl.bl_logprobs(st["x"], st["target"], scale=c["scale"], workspace=st["workspace"], **o)
    dx = bl.bl_logprobs_backward(st["x"], st["target"], o["lse"], o["entropy"], st["gl"], dentropy=st["gh"], dlse=st["gz"],
                                 scale=c["scale"], dlogits=st["dx"])
    return [o["logprob"], o["entropy"], dx]


def _copied(caches, copies):
    """(source, page, tokens) rows, -1 where there is nothing to do."""
    todo = copies[copies[:, 0] >= 0].long()
    if not todo.numel():
        return
    for k, v, ka, va in caches:
        fresh = (torch.arange(k.shape[2], device=DEV) < todo[:, 2:3])[:, None, :, None]
        for codes in (k, v):
            codes[todo[:, 1]] = torch.where(fresh, codes[todo[:, 0]], codes[todo[:, 1]])
        for a in (ka, va):
            a[todo[:, 1]] = a[todo[:, 0]]


def _handed(refs, need, short):
    """Free pages, lowest first, for the requests in order (-1: none left)."""
    free = torch.nonzero(refs == 0)[:, 0]
    rank = torch.cumsum(need.flatten().long(), 0) - 1
    got = need.flatten() & (rank < free.numel())
    pages = torch.full(rank.shape, -1, dtype=torch.int64, device=DEV)
    pages[got] = free[rank[got]]
    refs[pages[got]] = 1
    short += (need.sum() - got.sum()).int()
    return pages.view(need.shape)


def _plain_fork(st, c):
    page, refs, table, n = c["page"], st["refs"], st["table"].long(), c["children"]
    refs.copy_(st["refs0"])
    short = torch.zeros(1, dtype=torch.int32, device=DEV)
    parent = st["parent"].long()
    length = st["length"][parent]
    full, part = length.long() // page, length.long() % page
    column, child = torch.arange(table.shape[1], device=DEV), torch.arange(n, device=DEV)
    whole = column < full[:, None]
    rows = table[parent]
    out = torch.where(whole, rows, -1)
    first = torch.full((c["seqs"],), n, device=DEV).scatter_reduce_(0, parent, child, "amin")
    stays = (part > 0) & (first[parent] == child) & c["consume"]
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    need = (part > 0) & ~stays
    fresh = _handed(refs, need, short)
    out[child[part > 0], full[part > 0]] = torch.where(stays, last, fresh)[part > 0]
    one = torch.ones((), dtype=torch.int32, device=DEV)
    refs.index_add_(0, out[whole], one.expand(int(whole.sum())))
    if c["consume"]:
        refs.index_add_(0, last[stays], one.expand(int(stays.sum())))
        gone = table[table >= 0]
        refs.index_add_(0, gone, -one.expand(gone.numel()))
    did = need & (fresh >= 0)
    copies = torch.where(did[:, None], torch.stack([last, fresh, part], 1), torch.tensor([-1, -1, 0], device=DEV)).int()
    _copied(st["caches"], copies)
    # pages for the new tokens
    index = length.long()[:, None] // page + torch.arange((c["new"] + page - 2) // page + 1, device=DEV)
    inside = index * page < (length.long() + c["new"])[:, None]
    held = out.gather(1, index.clamp(max=table.shape[1] - 1))
    need = inside & (held < 0)
    fresh = _handed(refs, need, short)
    out[child[:, None].expand(index.shape)[need], index[need]] = fresh[need]
    return [refs, out.int(), length, copies, short] + [t for cache in st["caches"] for t in cache]


def _plain_compact(st, c):
    page, refs, table = c["page"], st["refs"], st["table"]
    refs.copy_(st["refs0"])
    table.copy_(st["table0"])
    left = (st["keep"].long() + page - 1) // page
    gone = (torch.arange(table.shape[1], device=DEV) >= left[:, None]) & (table >= 0)
    pages = table[gone].long()
    refs.index_add_(0, pages, torch.full(pages.shape, -1, dtype=torch.int32, device=DEV))
    table[gone] = -1
    used = refs > 0
    count = int(used.sum())
    to = torch.nonzero(~used[:count])[:, 0]
    source = torch.nonzero(used[count:])[:, 0].flip(0) + count  # the highest first
    moved = min(to.numel(), st["moves"])
    to, source = to[:moved], source[:moved]
    name = torch.arange(refs.numel(), device=DEV)
    name[source] = to
    table.copy_(torch.where(table >= 0, name[table.clamp(min=0).long()].int(), table))
    refs[to], refs[source] = refs[source], 0
    copies = torch.tensor([-1, -1, 0], dtype=torch.int32, device=DEV).repeat(st["moves"], 1)
    copies[:moved] = torch.stack([source, to, torch.full_like(to, page)], 1).int()
    _copied(st["caches"], copies)
    return [refs, table, copies, torch.full((1,), moved, dtype=torch.int32, device=DEV)] + [t for cache in st["caches"] for t in cache]


def _plain_shared(st, c):
    heads, dim, page, width = c["hkv"], c["dim"], c["page"], c["width"]
    group, out = c["hq"] // heads, torch.empty(st["total"], c["hq"], dim, dtype=BF16, device=DEV)
    prefix, ctx, new = _answers(c)  # a program knows its lengths
    begin = 0

    def values(codes, a, ids):  # [heads, tokens, dim]
        return (codes[ids].float() * (a[ids] / 127.0)[..., None, None]).transpose(0, 1).reshape(heads, -1, dim)

    for g, p in enumerate(prefix):
        mine = range(g * width, (g + 1) * width)
        total = sum(new[s] for s in mine)
        q = st["q"][begin:begin + total].float().view(total, heads, group, dim).permute(1, 0, 2, 3).reshape(heads, -1, dim)
        ids = st["table"][g * width].long()
        early = torch.matmul(q, values(st["kc"], st["ka"], ids[:p // page]).transpose(1, 2).contiguous()).mul_(1.0 / math.sqrt(dim))
        top = early.amax(dim=2)
        early = early.sub_(top[..., None]).exp_()
        sums = early.sum(dim=2)
        o = torch.matmul(early, values(st["vc"], st["va"], ids[:p // page]))
        at = 0
        for s in mine:
            n, a = new[s], ctx[s]
            rows = slice(at * group, (at + n) * group)
            ids = st["table"][s, p // page:-(-(p + a + n) // page)].long()
            k, v = values(st["kc"], st["ka"], ids)[:, :a + n], values(st["vc"], st["va"], ids)[:, :a + n]
            late = torch.matmul(q[:, rows], k.transpose(1, 2).contiguous()).mul_(1.0 / math.sqrt(dim)).view(heads, n, group, a + n)
            seen = torch.arange(a + n, device=DEV) <= a + torch.arange(n, device=DEV)[:, None]
            late = late.masked_fill(~seen[:, None], -math.inf).view(heads, n * group, a + n)
            most = torch.maximum(top[:, rows], late.amax(dim=2))
            late = (late - most[..., None]).exp()
            keep = (top[:, rows] - most).exp()
            r = (o[:, rows] * keep[..., None] + torch.matmul(late, v)) / (sums[:, rows] * keep + late.sum(dim=2))[..., None]
            out[begin + at:begin + at + n] = r.view(heads, n, group, dim).permute(1, 0, 2, 3).reshape(n, c["hq"], dim).to(BF16)
            at += n
        begin += total
    return out


def _stats(x, c):
    z = x.float() * c["scale"]
    top = z.amax(dim=1, keepdim=True)
    d = z - top
    e = d.exp()
    s = e.sum(dim=1)
    entropy = s.log() - (e * d.clamp(min=-1e4)).sum(dim=1) / s
    return z, top[:, 0] + s.log(), top[:, 0], s, entropy


def _chosen(z, target, lse):
    known = target >= 0
    z = z.gather(1, target.clamp(min=0).long()[:, None])[:, 0]
    return torch.where(known, z - lse, torch.zeros((), device=DEV))


def _plain_logprobs(st, c):
    x, n = st["x"], c["n"]
    z, lse, _, _, entropy = _stats(x, c)
    out = [_chosen(z, st["target"], lse), lse, entropy]
    if c["top"]:
        t = min(c["top"], n)
        bits = (x.float() + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()  # integers that order like the values
        ids = n - 1 - (torch.topk(order * n + (n - 1 - torch.arange(n, device=DEV)), t, dim=1).values % n)
        value = z.gather(1, ids)
        there = value > -math.inf
        top_id = torch.full((c["m"], c["top"]), -1, dtype=torch.int32, device=DEV)
        top_logprob = torch.full((c["m"], c["top"]), -math.inf, device=DEV)
        top_id[:, :t] = torch.where(there, ids, -1).int()
        top_logprob[:, :t] = torch.where(there, value - lse[:, None], -math.inf)
        out += [top_id, top_logprob]
    return out


def _plain_train(st, c):
    z, lse, top, s, entropy = _stats(st["x"], c)
    logprob = _chosen(z, st["target"], lse)
    known = (st["target"] >= 0).float()
    log_p = (z - top[:, None]) - s.log()[:, None]
    p = log_p.exp()
    slope = (st["gz"] - st["gl"] * known)[:, None] * p
    slope -= st["gh"][:, None] * p * (log_p.clamp(min=-1e4) + entropy[:, None])
    slope.scatter_add_(1, st["target"].clamp(min=0).long()[:, None], (st["gl"] * known)[:, None])
    return [logprob, entropy, (slope * c["scale"]).to(st["x"].dtype)]


_OWN = {"fork": _own_fork, "compact": _own_compact, "shared": _own_shared, "logprobs": _own_logprobs, "train": _own_train}
_PLAIN = {"fork": _plain_fork, "compact": _plain_compact, "shared": _plain_shared, "logprobs": _plain_logprobs,
          "train": _plain_train}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    st, c = prepare(case, seed), case
    return {"fork": _exact_fork, "compact": _exact_compact, "shared": _exact_shared, "logprobs": _exact_logprobs,
            "train": _exact_train}[c["op"]](st, c)


def _moved_caches(st, copies):
    """Page by page, in order (nothing that is written is read again)."""
    for source, to, n in copies:
        if source >= 0:
            for k, v, ka, va in st["caches"]:
                for codes in (k, v):
                    codes[to, :, :n] = codes[source, :, :n]
                for a in (ka, va):
                    a[to] = a[source]
    return [t.double() if t.is_floating_point() else t for cache in st["caches"] for t in cache]


def _exact_fork(st, c):
    page, refs, table = c["page"], st["refs0"].tolist(), st["table0"].tolist()
    length, parent = st["length"].tolist(), st["parent"].tolist()
    free = [p for p, r in enumerate(refs) if r == 0][::-1]
    rows, copies, stayed = [], [], set()
    for p in parent:
        n, rest = length[p] // page, length[p] % page
        row, copy = table[p][:n], (-1, -1, 0)
        if rest and c["consume"] and p not in stayed:
            row = row + [table[p][n]]
        elif rest:
            copy = (table[p][n], free.pop(), rest)
            row = row + [copy[1]]
        stayed.add(p)
        rows.append(row)
        copies.append(copy)
    held = rows + ([] if c["consume"] else [[p for p in r if p >= 0] for r in table])

    def count():
        n = [0] * len(refs)
        for r in held:
            for p in r:
                n[p] += 1
        return n

    free = [p for p, r in enumerate(count()) if r == 0][::-1]
    for row, p in zip(rows, parent):
        while len(row) * page < length[p] + c["new"]:
            row.append(free.pop())
    stride = len(table[0])
    return [_ints(count()), _ints([r + [-1] * (stride - len(r)) for r in rows]), _ints([length[p] for p in parent]),
            _ints(copies), _ints([0])] + _moved_caches(st, copies)


def _exact_compact(st, c):
    page, keep = c["page"], st["keep"].tolist()
    rows = [r[:-(-n // page)] for r, n in zip(st["table0"].tolist(), keep)]
    pages = len(st["refs0"])
    held = {p for r in rows for p in r}
    above, below = sorted((p for p in held if p >= len(held)), reverse=True), [p for p in range(len(held)) if p not in held]
    copies = [(a, b, page) for a, b in zip(above, below)]
    name = {a: b for a, b, _ in copies}
    rows = [[name.get(p, p) for p in r] for r in rows]
    refs = [0] * pages
    for r in rows:
        for p in r:
            refs[p] += 1
    stride = st["table0"].shape[1]
    return [_ints(refs), _ints([r + [-1] * (stride - len(r)) for r in rows]),
            _ints(copies + [(-1, -1, 0)] * (st["moves"] - len(copies))) if st["moves"] else torch.empty(0, 3, dtype=torch.int32),
            _ints([len(copies)])] + _moved_caches(st, copies)


def _exact_shared(st, c):
    """Each sequence by itself, over its whole row of pages."""
    group, start, offsets, out = c["hq"] // c["hkv"], st["start"].tolist(), st["offsets"].tolist(), []
    for s, a in enumerate(start):
        n = offsets[s + 1] - offsets[s]
        ids = st["table"][s, :-(-(a + n) // c["page"])].long()
        parts = []
        for h in range(c["hkv"]):
            k, v = ((codes[ids, h].double() * (top[ids, h].double() / 127.0)[:, None, None]).flatten(0, 1)[:a + n]
                    for codes, top in ((st["kc"], st["ka"]), (st["vc"], st["va"])))
            rows = []
            for lo in range(0, n, 512):
                at = torch.arange(a + lo, a + min(n, lo + 512), device=DEV)[:, None]
                q = st["q"][offsets[s] + lo:offsets[s] + lo + at.shape[0], h * group:(h + 1) * group].double()
                score = torch.matmul(q.transpose(0, 1), k.T.contiguous()) / math.sqrt(c["dim"])
                p = torch.softmax(score.masked_fill(torch.arange(a + n, device=DEV) > at, -math.inf), dim=-1)
                rows.append(torch.matmul(p, v).transpose(0, 1))
            parts.append(torch.cat(rows))
        out.append(torch.cat(parts, dim=1))
    return torch.cat(out)


def _exact_rows(st, c):
    """Row blocks: (first row, log probabilities, log of the sum, entropy, target's log probability)."""
    rows = max(1, (1 << 26) // c["n"])
    for lo in range(0, c["m"], rows):
        z = st["x"][lo:lo + rows].double() * c["scale"]
        lse = torch.logsumexp(z, dim=1)
        log_p = z - lse[:, None]
        p = log_p.exp()
        entropy = -torch.where(p > 0, p * log_p, 0.0).sum(dim=1)
        target = st["target"][lo:lo + rows].long()
        chosen = torch.where(target >= 0, log_p.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
        yield lo, log_p, p, lse, entropy, chosen, target


def _exact_logprobs(st, c):
    parts = []
    for lo, log_p, _, lse, entropy, chosen, _ in _exact_rows(st, c):
        part = [chosen, lse, entropy]
        if c["top"]:
            x = st["x"][lo:lo + log_p.shape[0]].double()
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
            value = log_p.gather(1, ids)
            ids = torch.where(torch.isinf(value), -1, ids)
            lack = c["top"] - ids.shape[1]
            part += [torch.nn.functional.pad(ids, (0, lack), value=-1).int(),
                     torch.nn.functional.pad(value, (0, lack), value=-math.inf)]
        parts.append(part)
    return [torch.cat(v) for v in zip(*parts)]


def _exact_train(st, c):
    parts = []
    for lo, log_p, p, _, entropy, chosen, target in _exact_rows(st, c):
        gl, gh, gz = (st[k][lo:lo + p.shape[0], None].double() for k in ("gl", "gh", "gz"))
        hit = torch.zeros_like(p).scatter_(1, target.clamp(min=0)[:, None], 1.0)
        scored = (target >= 0)[:, None].double()
        of_entropy = torch.where(p > 0, p * (log_p + entropy[:, None]), 0.0)
        parts.append([chosen, entropy, c["scale"] * (gl * scored * (hit - p) - gh * of_entropy + gz * p)])
    return [torch.cat(v) for v in zip(*parts)]
