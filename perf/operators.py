"""What the paged key-value cache and the attention that reads it are measured on.

Four operators of the serving path, between a layer's q/k/v projections and its output projection:

* append   new tokens' keys and values (fp32 or fp16 rows) into the pages of a cache held in fp16 or
           in E4M3 with a power-of-two scale for each token and head
* decode   attention of one new token of each sequence over its pages, with an optional sliding window
           whose first tokens (sinks) stay visible
* prompt   the same attention for many new tokens of each sequence, a ragged batch, over pages that
           already hold them
* pages    the pages themselves: sequences freed, forked and grown; the pool compacted; pages copied

The plain forms below are elementary torch operations in fp32 (the exact ones in fp64).
"""
import math
import random

import torch

own = False

FP16_MAX = 65504.0
SCALE_MIN, SCALE_MAX = -15, 8  # exponents of an E4M3 row's scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one chat of a few hundred tokens at the LLaMA-7B head layout: latency counts
        dict(name="decode_one", op="decode", e4m3=False, heads=32, kv=32, dim=128, page=16, n=1, lo=333, hi=333, window=0,
             sinks=0, mix=1),
        # a serving batch of unlike lengths with shared key-value heads (LLaMA-2-70B's layout)
        dict(name="decode_ragged", op="decode", e4m3=False, heads=64, kv=8, dim=128, page=16, n=64, lo=0, hi=8191, window=0,
             sinks=0, mix=2),
        # long chats under a sliding window with sinks, an 8-bit cache
        dict(name="decode_window", op="decode", e4m3=True, heads=32, kv=32, dim=128, page=32, n=32, lo=2000, hi=32768,
             window=4096, sinks=4, mix=3),
        # one very long document: the work has to be split over its length
        dict(name="decode_long", op="decode", e4m3=True, heads=64, kv=8, dim=128, page=64, n=1, lo=250001, hi=250001, window=0,
             sinks=0, mix=4),
        # short prompts at the BERT-base head layout, ragged
        dict(name="prompt_short", op="prompt", e4m3=False, heads=12, kv=12, dim=64, page=16, n=5, lo=17, hi=333, qlo=17, qhi=333,
             window=0, sinks=0, mix=5),
        # a chunk of a long prompt over an 8-bit cache, sliding window and sinks, shared heads
        dict(name="prompt_chunk", op="prompt", e4m3=True, heads=64, kv=8, dim=128, page=64, n=2, lo=12000, hi=16384, qlo=1000,
             qhi=2048, window=4096, sinks=4, mix=6),
        # whole long prompts, causal
        dict(name="prompt_long", op="prompt", e4m3=False, heads=32, kv=32, dim=128, page=128, n=2, lo=8192, hi=8192, qlo=8192,
             qhi=8192, window=0, sinks=0, mix=7),
        # one decode step's rows, straight from the projections (fp32), into an 8-bit cache
        dict(name="append_step", op="append", e4m3=True, f32=True, kv=8, dim=128, page=16, n=64, lo=1, hi=2000, qlo=1, qhi=1,
             mix=8),
        # prompts' rows into an fp16 cache
        dict(name="append_prompt", op="append", e4m3=False, f32=True, kv=32, dim=128, page=16, n=7, lo=900, hi=4096, qlo=900,
             qhi=2048, mix=9),
        # parallel sampling: the last step's branches are dropped, forked again and grown
        dict(name="pages_fork", op="pages", do="fork", e4m3=False, kv=8, dim=128, page=16, layers=4, n=4, lo=100, hi=3000,
             children=16, grow=40, mix=10),
        # a fragmented pool made dense
        dict(name="pages_compact", op="pages", do="compact", e4m3=True, kv=8, dim=128, page=64, layers=8, n=48, lo=1, hi=1500,
             spread=0.6, mix=11),
        # prefixes brought from one pool into another
        dict(name="pages_copy", op="pages", do="copy", e4m3=False, kv=32, dim=128, page=16, layers=2, pool=1500, copies=777,
             mix=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "append", "pages", "pages"])
    kv = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])
    group = rng.choice([g for g in (1, 1, 2, 3, 4, 5, 7, 8, 16) if g * kv <= 64])
    case = dict(op=op, e4m3=rng.random() < 0.5, kv=kv, dim=rng.choice([64, 128, 128, 32, 40, 80, 96, 112]),
                page=rng.choice([16, 16, 32, 48, 64, 128, 256]), mix=rng.randrange(1 << 30))
    if op in ("decode", "prompt"):
        case["heads"] = kv * group
        case["window"] = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        case["sinks"] = rng.choice([0, rng.randint(1, 200)]) if case["window"] else 0
    if op == "decode":
        case["n"] = _log_int(rng, 1, 200)
        case["hi"] = _log_int(rng, 1, 60000)
        case["lo"] = rng.choice([0, case["hi"] // 2, case["hi"]])
    elif op == "prompt":
        case["n"] = _log_int(rng, 1, 16)
        case["qhi"] = _log_int(rng, 1, 8192)
        case["qlo"] = rng.choice([1, case["qhi"] // 2 + 1, case["qhi"]])
        case["lo"] = case["qhi"]
        case["hi"] = case["qhi"] + rng.choice([0, _log_int(rng, 1, 8192)])
    elif op == "append":
        case["f32"] = rng.random() < 0.5
        case["n"] = _log_int(rng, 1, 128)
        case["qhi"] = _log_int(rng, 1, 2048)
        case["qlo"] = rng.choice([1, case["qhi"]])
        case["lo"], case["hi"] = case["qhi"], case["qhi"] + rng.randint(0, 2000)
    else:
        case["do"] = rng.choice(["fork", "compact", "copy"])
        case["layers"] = rng.randint(1, 8)
        if case["do"] == "copy":
            case["pool"] = _log_int(rng, 8, 2000)
            case["copies"] = rng.randint(1, case["pool"])
        else:
            case["n"] = rng.randint(1, 24)
            case["hi"] = _log_int(rng, 2, 4000)
            case["lo"] = 1
            if case["do"] == "fork":
                case["children"], case["grow"] = rng.randint(1, 48), rng.randint(1, 100)
            else:
                case["spread"] = round(rng.uniform(0.2, 0.95), 3)
    while _size(case) > 1 << 28 or work(case)["flops"] > 6e11:  # a drawn case stays below the largest listed one
        if "n" in case and case["n"] > 1:
            case["n"] //= 2
        elif "pool" in case:
            case["pool"] //= 2
            case["copies"] = max(1, case["copies"] // 2)
        elif case.get("layers", 1) > 1:
            case["layers"] //= 2
        else:
            for k in ("lo", "hi", "qlo", "qhi"):
                if case.get(k, 0) > 1:
                    case[k] = (case[k] + 1) // 2
    return case


# ------------------------------------------------------------------ geometry, from the case alone
def _lens(case):
    """(tokens in the cache after this step, new tokens) of each sequence."""
    r = random.Random(case["mix"])
    new, total = [], []
    for _ in range(case["n"]):
        q = r.randint(case["qlo"], case["qhi"]) if "qlo" in case else 1
        t = r.randint(case["lo"], case["hi"])
        total.append(max(t, q) if "qlo" in case else t)
        new.append(q)
    return total, new


def _pages(n, case):
    return -(-n // case["page"])


def _need(case):
    """Pages in use, and the longest row of pages."""
    if case.get("do") == "copy":
        return case["pool"], 1
    total, _ = _lens(case)
    used, most = sum(_pages(t, case) for t in total), max(_pages(t, case) for t in total)
    if case.get("do") == "fork":
        grown = max(total) + case["grow"]
        return used + case["children"] * (_pages(case["grow"], case) + 2), _pages(grown, case)
    return used, most


def _pool(case):
    used, _ = _need(case)
    if case.get("do") == "copy":
        return used
    if case.get("do") == "compact":
        return max(used + 1, int(used / case["spread"]))
    return used + 3


def _size(case):
    return _pool(case) * case["page"] * case["kv"] * case["dim"] * case.get("layers", 1) * (1 if case["e4m3"] else 2)


def _page_bytes(case):
    """Keys, values and scales of one page in one layer."""
    return 2 * case["page"] * case["kv"] * (case["dim"] + 4 if case["e4m3"] else 2 * case["dim"])


def _visible(p, case):
    """How many keys the query at position p sees."""
    w, s = case["window"], case["sinks"]
    if not w or p + 1 <= w:
        return p + 1
    return w + min(s, p + 1 - w)


def work(case):
    d, kv, elt = case["dim"], case["kv"], (1 if case["e4m3"] else 2)
    row = 2 * kv * (d * elt + (4 if case["e4m3"] else 0))  # one token's keys and values
    if case["op"] == "decode":
        total, _ = _lens(case)
        keys = sum(_visible(t - 1, case) for t in total if t)
        io = 2 * 2 * case["n"] * case["heads"] * d + 4 * sum(_pages(t, case) for t in total)
        return {"bytes": keys * row + io, "flops": 4 * d * case["heads"] * keys}
    if case["op"] == "prompt":
        total, new = _lens(case)
        pairs = seen = 0
        for t, q in zip(total, new):
            w, s = case["window"], case["sinks"]
            pairs += q * (2 * t - q + 1) // 2 if not w else sum(_visible(p, case) for p in range(t - q, t))
            first = max(0, t - q - w + 1) if w else 0
            seen += t - first + min(s, first)
        return {"bytes": seen * row + 2 * 2 * sum(new) * case["heads"] * d, "flops": 4 * d * case["heads"] * pairs}
    if case["op"] == "append":
        total, new = _lens(case)
        return {"bytes": sum(new) * (2 * kv * d * (4 if case["f32"] else 2) + row), "flops": 2 * sum(new) * kv * d * (2 if case["e4m3"] else 1)}
    if case["do"] == "copy":
        return {"bytes": 2 * case["copies"] * case["layers"] * _page_bytes(case), "flops": 0}
    total, _ = _lens(case)
    if case["do"] == "fork":
        partial = rows = 0
        for c in range(case["children"]):
            t = total[c % case["n"]]
            partial += t % case["page"] != 0
            rows += _pages(t, case) + _pages(t + case["grow"], case)
        moved = 2 * partial * case["layers"] * _page_bytes(case)
        return {"bytes": moved + 4 * 4 * rows + 4 * _pool(case), "flops": 0}
    owner, _, _ = _scatter(case)
    used = sum(p >= 0 for p in owner)
    far = sum(p >= 0 for p in owner[used:])
    return {"bytes": 2 * far * case["layers"] * _page_bytes(case) + 4 * (2 * used + len(owner)), "flops": 0}


def _scatter(case):
    """A pool's pages dealt to the sequences in a random order: (owner of each page, rows of pages, lengths)."""
    total, _ = _lens(case)
    pool = _pool(case)
    order = list(range(pool))
    random.Random(case["mix"] + 1).shuffle(order)
    owner, rows, at = [-1] * pool, [], 0
    for s, t in enumerate(total):
        k = _pages(t, case)
        rows.append(order[at:at + k])
        at += k
        for p in rows[-1]:
            owner[p] = s
    return owner, rows, total


# ------------------------------------------------------------------ inputs
class _Bag(dict):
    __getattr__ = dict.__getitem__


def _fill_cache(case, g, pool):
    """One layer's pool as a running program holds it: [pages][heads][page][dim], fp16, or E4M3 bytes with scales."""
    shape = (pool, case["kv"], case["page"], case["dim"])
    got = []
    for shift in (0.0, 0.25):  # keys; values, off zero
        x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(shift, 1.0, generator=g)
        if not case["e4m3"]:
            got += [x, None]
            continue
        e = torch.randint(-9, -6, shape[:3], device="cuda", generator=g).float()
        codes = (x.float() * torch.exp2(-e)[..., None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        got += [codes.view(torch.uint8), torch.exp2(e)]
    return _Bag(k=got[0], k_scale=got[1], v=got[2], v_scale=got[3])


def _own_cache(c):
    import binarized_transformer_b200 as bt
    return bt.KvCache(c.k, c.v, c.k_scale, c.v_scale)


def _own_table(t):
    import binarized_transformer_b200 as bt
    return bt.KvTable(t.pages, t.kv_len, t.refcount)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(case, extra=0):
    owner, rows, total = _scatter(case)
    _, most = _need(case)
    pages = torch.full((len(rows) + extra, most), -1, dtype=torch.int32)
    for s, r in enumerate(rows):
        pages[s, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return _Bag(pages=pages.cuda(), kv_len=_ints(total + [0] * extra), refcount=_ints([int(o >= 0) for o in owner])), total


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = _Bag(case=case)
    if case["op"] == "pages":
        _prepare_pages(st, case, g)
    else:
        st["cache"] = _fill_cache(case, g, _pool(case))
        st["table"], st["total"] = _table(case)
        _, st["new"] = _lens(case)
        at = [0]
        for q in st.new:
            at.append(at[-1] + q)
        st["at"], st["cu_q"] = at, _ints(at)
        st["step"] = all(q == 1 for q in st.new)
        rows = at[-1]
        if case["op"] == "append":
            shape, kind = (rows, case["kv"], case["dim"]), torch.float32 if case["f32"] else torch.float16
            # activations: heads of unlike sizes, a few outliers
            size = torch.exp(torch.randn(shape[1], 1, device="cuda", generator=g))
            for name in ("k", "v"):
                x = torch.randn(shape, device="cuda", generator=g) * size
                x = torch.where(torch.rand(shape, device="cuda", generator=g) < 0.01, x * 20, x)
                st[name] = x.to(kind)
        else:
            st["scale"] = case["dim"] ** -0.5
            st["q"] = torch.randn((rows, case["heads"], case["dim"]), device="cuda", generator=g).half()
        if own:
            st["ocache"], st["otable"] = _own_cache(st.cache), _own_table(st.table)
    return st


def _prepare_pages(st, case, g):
    st["caches"] = [_fill_cache(case, g, _pool(case)) for _ in range(case["layers"])]
    if case["do"] == "copy":
        st["into"] = [_fill_cache(case, g, _pool(case)) for _ in range(case["layers"])]
        st["src"] = torch.randperm(case["pool"], device="cuda", generator=g)[:case["copies"]].int()
        st["dst"] = torch.randperm(case["pool"], device="cuda", generator=g)[:case["copies"]].int()
    else:
        st["table"], total = _table(case, case.get("children", 0))
        if case["do"] == "fork":
            st["src"] = _ints([c % case["n"] for c in range(case["children"])])
            st["dst"] = _ints([case["n"] + c for c in range(case["children"])])
            st["grow"] = _ints([case["grow"]] * case["children"])
            _fork(st.caches, st.table, st.src, st.dst, case["page"])
            _reserve(st.table, st.dst, st.grow, case["page"])
        else:
            st["saved"] = (st.table.pages.clone(), st.table.refcount.clone())
    if own:
        import binarized_transformer_b200 as bt
        st["ocaches"] = bt.kv_layers([_own_cache(c) for c in st.caches])
        if case["do"] == "copy":
            st["ointo"] = bt.kv_layers([_own_cache(c) for c in st.into])
        else:
            st["otable"] = _own_table(st.table)


# ------------------------------------------------------------------ one pass
def run(st):
    case = st.case
    if case["op"] == "decode":
        if own:
            import binarized_transformer_b200 as bt
            return bt.bwta_attn_decode_paged(st.q, st.ocache, st.otable, st.scale, window=case["window"], sinks=case["sinks"])
        return _attention(st, torch.float32).half()
    if case["op"] == "prompt":
        if own:
            import binarized_transformer_b200 as bt
            return bt.bwta_attn_prompt_paged(st.q, st.cu_q, st.ocache, st.otable, st.scale, window=case["window"],
                                             sinks=case["sinks"])
        return _attention(st, torch.float32).half()
    if case["op"] == "append":
        if own:
            import binarized_transformer_b200 as bt
            bt.bwta_kv_append(st.ocache, st.otable, st.k, st.v, cu_q=None if st.step else st.cu_q)
        else:
            _append(st)
        return _whole([st.cache])
    if case["do"] == "copy":
        if own:
            import binarized_transformer_b200 as bt
            bt.bwta_kv_copy_pages(st.ocaches, st.ointo, st.src, st.dst)
        else:
            s, d = st.src.long(), st.dst.long()
            for a, b in zip(st.caches, st.into):
                for name in ("k", "v", "k_scale", "v_scale"):
                    if a[name] is not None:
                        b[name][d] = a[name][s]
        return _whole(st.into)
    if case["do"] == "fork":
        if own:
            import binarized_transformer_b200 as bt
            bt.bwta_kv_free(st.otable, case["page"], st.dst)
            bt.bwta_kv_fork(st.ocaches, st.otable, st.src, st.dst)
            bt.bwta_kv_reserve(st.otable, case["page"], st.dst, st.grow)
        else:
            _free(st.table, st.dst, case["page"])
            _fork(st.caches, st.table, st.src, st.dst, case["page"])
            _reserve(st.table, st.dst, st.grow, case["page"])
        return _whole(st.caches) + [st.table.pages, st.table.kv_len, st.table.refcount]
    st.table.pages.copy_(st.saved[0])  # fragmented again, as the requests that ended since would leave it
    st.table.refcount.copy_(st.saved[1])
    if own:
        import binarized_transformer_b200 as bt
        live = bt.bwta_kv_compact(st.ocaches, st.otable)
    else:
        live = _compact(st.caches, st.table, case["page"])
    return _whole(st.caches) + [st.table.pages, st.table.refcount, live]


def _whole(caches):
    """The pools' values: 8-bit ones as the E4M3 numbers that the bytes are, beside their scales."""
    out = []
    for c in caches:
        for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
            out += [x] if s is None else [x.view(torch.float8_e4m3fn), s]
    return out


# ------------------------------------------------------------------ plain forms
def _gathered(st, s, kind):
    """Keys and values of sequence s, [heads][tokens][dim]."""
    c, page, t = st.cache, st.case["page"], st.total[s]
    rows = st.table.pages[s, :_pages(t, st.case)].long()
    got = []
    for x, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        y = x[rows]
        if sc is not None:
            y = y.view(torch.float8_e4m3fn).to(kind) * sc[rows].to(kind)[..., None]
        got.append(y.to(kind).transpose(0, 1).reshape(st.case["kv"], -1, st.case["dim"])[:, :t])
    return got


def _attention(st, kind):
    case, out = st.case, torch.zeros_like(st.q, dtype=kind)
    group = case["heads"] // case["kv"]
    for s, (t, n) in enumerate(zip(st.total, st.new)):
        if t == 0:
            continue
        k, v = _gathered(st, s, kind)
        key = torch.arange(t, device="cuda")
        step = max(1, (1 << 28) // (t * group))  # queries at a time
        for a in range(0, n, step):
            b = min(n, a + step)
            pos = torch.arange(t - n + a, t - n + b, device="cuda")[:, None]
            seen = key <= pos
            if case["window"]:
                seen &= (key > pos - case["window"]) | (key < case["sinks"])
            for h in range(case["kv"]):
                q = st.q[st.at[s] + a:st.at[s] + b, h * group:(h + 1) * group].to(kind).transpose(0, 1)
                x = ((q @ k[h].T) * st.scale).masked_fill_(~seen, -math.inf)
                e = x.sub_(x.amax(-1, keepdim=True)).exp_()
                o = (e @ v[h]) / e.sum(-1, keepdim=True)
                out[st.at[s] + a:st.at[s] + b, h * group:(h + 1) * group] = o.transpose(0, 1)
    return out


def _quantized(x):
    """Rows of fp32 as E4M3 bytes and the smallest power of two that brings them within 448."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).int()).clamp(SCALE_MIN, SCALE_MAX)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    most = torch.where(e == SCALE_MAX, 240.0, 448.0)[..., None]  # 256 * 2^8 would pass the largest fp16
    y = torch.ldexp(x, -e[..., None])
    return torch.minimum(torch.maximum(y, -most), most).to(torch.float8_e4m3fn).view(torch.uint8), torch.ldexp(torch.ones_like(top), e)


def _append(st):
    c, page = st.cache, st.case["page"]
    pos = torch.cat([torch.arange(t - n, t, device="cuda") for t, n in zip(st.total, st.new)])
    seq = torch.repeat_interleave(torch.arange(len(st.new), device="cuda"), torch.tensor(st.new, device="cuda"))
    at = (st.table.pages[seq, pos // page].long(), slice(None), pos % page)
    for x, to, scale in ((st.k, c.k, c.k_scale), (st.v, c.v, c.v_scale)):
        if scale is None:
            to[at[0], :, at[2]] = x.half()
        else:
            codes, sc = _quantized(x.float())
            to[at[0], :, at[2]] = codes
            scale[at[0], :, at[2]] = sc


def _owned(table, slots, page):
    """The pages that these slots hold, as a mask over their rows."""
    have = (table.kv_len[slots] + page - 1) // page
    return torch.arange(table.pages.shape[1], device="cuda") < have[:, None]


def _free(table, slots, page):
    slots = slots.long()
    mine = table.pages[slots][_owned(table, slots, page)].long()
    table.refcount.index_add_(0, mine, torch.full_like(mine, -1, dtype=torch.int32))
    table.pages[slots] = -1
    table.kv_len[slots] = 0


def _fork(caches, table, src, dst, page):
    src, dst = src.long(), dst.long()
    length = table.kv_len[src]
    rows = torch.where(_owned(table, src, page), table.pages[src], -1)
    full = torch.arange(rows.shape[1], device="cuda") < (length // page)[:, None]
    mine = rows[full].long()
    who = torch.nonzero(length % page).reshape(-1)  # their last page is not full: a copy of their own
    new = torch.nonzero(table.refcount == 0).reshape(-1)[:len(who)]
    table.refcount.index_add_(0, mine, torch.ones_like(mine, dtype=torch.int32))
    last = (length // page)[who].long()
    old = rows[who, last].long()
    for c in caches:
        for name in ("k", "v", "k_scale", "v_scale"):
            if c[name] is not None:
                c[name][new] = c[name][old]
    rows[who, last] = new.int()
    table.refcount[new] = 1
    table.pages[dst] = rows
    table.kv_len[dst] = length


def _reserve(table, slots, grow, page):
    slots = slots.long()
    old = table.kv_len[slots]
    have, want = (old + page - 1) // page, (old + grow + page - 1) // page
    at = torch.arange(table.pages.shape[1], device="cuda")
    fresh = (at >= have[:, None]) & (at < want[:, None])
    who, where = torch.nonzero(fresh, as_tuple=True)  # in the order of the slots, then of the row
    new = torch.nonzero(table.refcount == 0).reshape(-1)[:len(who)]
    table.pages[slots[who], where] = new.int()
    table.refcount[new] = 1
    table.kv_len[slots] = old + grow


def _compact(caches, table, page):
    used = table.refcount > 0
    live = used.sum()
    at = torch.arange(len(used), device="cuda")
    far, hole = torch.nonzero(used & (at >= live)).reshape(-1), torch.nonzero(~used & (at < live)).reshape(-1)
    for c in caches:
        for name in ("k", "v", "k_scale", "v_scale"):
            if c[name] is not None:
                c[name][hole] = c[name][far]
    to = at.clone()
    to[far] = hole
    slots = torch.arange(len(table.kv_len), device="cuda")
    mine = _owned(table, slots, page)
    table.pages[mine] = to[table.pages[mine].long()].int()
    table.refcount[hole] = table.refcount[far]
    table.refcount[far] = 0
    return live.int().reshape(1)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    if case["op"] == "pages":
        return None  # bytes and whole numbers are moved, nothing is computed
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attention(st)


def _exact_attention(st):
    case = st.case
    group = case["heads"] // case["kv"]
    out = torch.zeros(st.q.shape, dtype=torch.float64, device="cuda")
    for s in range(case["n"]):
        t, n = st.total[s], st.new[s]
        if t == 0:
            continue
        pos = torch.arange(t, device="cuda")
        place = st.table.pages[s].long()[pos // case["page"]], pos % case["page"]
        for h in range(case["kv"]):
            k = st.cache.k[place[0], h, place[1]]
            v = st.cache.v[place[0], h, place[1]]
            if case["e4m3"]:
                k = k.view(torch.float8_e4m3fn).double() * st.cache.k_scale[place[0], h, place[1]].double()[:, None]
                v = v.view(torch.float8_e4m3fn).double() * st.cache.v_scale[place[0], h, place[1]].double()[:, None]
            k, v = k.double(), v.double()
            for j in range(h * group, (h + 1) * group):
                for a in range(0, n, 2048):
                    i = torch.arange(t - n + a, t - n + min(n, a + 2048), device="cuda")[:, None]
                    sees = pos[None] <= i
                    if case["window"]:
                        sees = sees & ((i - pos[None] < case["window"]) | (pos[None] < case["sinks"]))
                    lo, hi = st.at[s] + a, st.at[s] + min(n, a + 2048)
                    z = torch.einsum("qd,kd->qk", st.q[lo:hi, j].double(), k) * case["dim"] ** -0.5
                    z = torch.where(sees, z, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                    p = torch.exp(z - z.max(1, keepdim=True).values)
                    out[lo:hi, j] = torch.einsum("qk,kd->qd", p / p.sum(1, keepdim=True), v)
    return out


def _exact_append(st):
    """Token by token's place; E4M3: nearest multiples of the step of each binade, ties to the even one."""
    case, c = st.case, st.cache
    kept = []
    for x, to, scale in ((st.k, c.k, c.k_scale), (st.v, c.v, c.v_scale)):
        x = x.double()
        vals = to.view(torch.float8_e4m3fn).double() if case["e4m3"] else to.double()
        sc = scale.double() if case["e4m3"] else None
        if case["e4m3"]:
            top = x.abs().amax(-1)
            e = torch.ceil(torch.log2(top / 448.0))
            e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, e)  # log2 rounds: the border settled by products
            e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e)
            e = torch.where(top == 0, torch.zeros_like(e), e.clamp(SCALE_MIN, SCALE_MAX))
            y = x / torch.exp2(e)[..., None]
            lim = torch.where(e == SCALE_MAX, 240.0, 448.0)[..., None].double()
            y = torch.minimum(torch.maximum(y, -lim), lim)
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
            y = torch.round(y / step) * step
        for s in range(case["n"]):
            p = torch.arange(st.total[s] - st.new[s], st.total[s], device="cuda")
            page = st.table.pages[s].long()[p // case["page"]]
            lo, hi = st.at[s], st.at[s + 1]
            vals[page, :, p % case["page"]] = y[lo:hi] if case["e4m3"] else x[lo:hi]
            if case["e4m3"]:
                sc[page, :, p % case["page"]] = torch.exp2(e)[lo:hi]
        kept += [vals, sc] if case["e4m3"] else [vals]
    return kept
