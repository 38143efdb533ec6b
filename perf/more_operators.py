"""Cases that measure the operators on a paged key/value cache in 16 bits, and their plain forms.

Four operators, in the order a serving process uses them:

* ``kv_write``    keys and values of new tokens into the cache's pages; their accumulated weights start at 0
* ``kv_attn``     attention of each sequence's newest tokens (one, or a chunk of a prompt) over its pages
* ``kv_weights``  the attention weight that each cached token got from those queries, summed over rows and heads
* ``kv_evict``    of each sequence and head the tokens with the largest weights stay, moved together in order

``run`` computes a case with elementary torch operations, or, where ``own`` is true, with the calls of
``ring_attention_slope_gb300``.

A cache holds keys [pages, heads, page size, dqk] and values [pages, heads, page size, dv] in bf16; a sequence's tokens
lie in the pages that its row of a block table lists.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    gqa = dict(Hq=64, Hkv=8, dqk=64, dv=64, page=64)
    return [
        # the new tokens of 32 decoding sequences, each into its own page: launch latency
        dict(name="kv_write_decode_32", op="kv_write", T=32, Hkv=8, dqk=64, dv=64, page=64, run=1, pad=0, wide=False),
        # one 12K prefill chunk into the cache's pages
        dict(name="kv_write_chunk_12k", op="kv_write", T=12288, Hkv=8, dqk=64, dv=64, page=64, run=64, pad=0,
             wide=False),
        # one sequence of a thousand tokens: the smallest decode step
        dict(name="kv_attn_1x1000", op="kv_attn", lens="equal", B=1, L=1000, new="one", chunk=1, window=0, **gqa),
        # a serving batch of single tokens with contexts from a few tokens to 32K
        dict(name="kv_attn_32x32k_ragged", op="kv_attn", lens="ragged", B=32, L=32768, new="one", chunk=1, window=0,
             **gqa),
        # a step that mixes the next chunk of one prompt with the decoding of fifteen sequences
        dict(name="kv_attn_mixed_16", op="kv_attn", lens="ragged", B=16, L=16384, new="mixed", chunk=1000, window=0,
             **gqa),
        # a 4K chunk of one long prompt
        dict(name="kv_attn_chunk_4k_at_64k", op="kv_attn", lens="equal", B=1, L=65536, new="each", chunk=4096, window=0,
             **gqa),
        # odd chunks of four prompts with wide heads, one query head for each key head, small pages
        dict(name="kv_attn_wide_4x777", op="kv_attn", lens="ragged", B=4, L=8192, new="each", chunk=777, window=0,
             Hq=32, Hkv=32, dqk=192, dv=128, page=16),
        # the weights of a decode step
        dict(name="kv_weights_16x8k", op="kv_weights", lens="equal", B=16, L=8192, new="one", chunk=1, window=0, **gqa),
        # the last 64 queries of two prompts look over the whole prompts
        dict(name="kv_weights_look_64", op="kv_weights", lens="ragged", B=2, L=32768, new="each", chunk=64, window=0,
             **gqa),
        # every query of a 2K chunk
        dict(name="kv_weights_chunk_2k_at_16k", op="kv_weights", lens="equal", B=1, L=16384, new="each", chunk=2048,
             window=0, **gqa),
        # one sequence of two thousand tokens down to 500
        dict(name="kv_evict_1x2000", op="kv_evict", lens="equal", B=1, L=2000, keep=500, first=4, recent=64, Hkv=8,
             dqk=64, dv=64, page=64),
        # four long contexts down to a quarter
        dict(name="kv_evict_4x64k", op="kv_evict", lens="ragged", B=4, L=65536, keep=16384, first=16, recent=1024,
             Hkv=8, dqk=64, dv=64, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv_write", "kv_attn", "kv_attn", "kv_attn", "kv_weights", "kv_weights", "kv_evict"])
    wide = rng.random() < 0.4
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * (rng.choice([1, 2, 3, 5, 8]) if wide else rng.choice([1, 4, 5, 7, 8, 8, 12]))
    dqk, dv = rng.choice([(128, 128), (192, 128), (128, 64), (64, 128)]) if wide else (64, 64)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "kv_write":
        T = _log(rng, 1, 12000)
        return dict(op=op, T=T, Hkv=Hkv, dqk=dqk, dv=dv, page=page, run=rng.choice([1, 5, page]),
                    pad=min(T - 1, rng.choice([0, 0, 3])), wide=rng.random() < 0.3)
    B = _log(rng, 1, 48)
    lens = rng.choice(["equal", "ragged"])
    if op == "kv_evict":
        L = max(40, min(_log(rng, 40, 65536), 200000 // B))
        keep = max(24, int(L * rng.uniform(0.1, 0.9)))
        return dict(op=op, lens=lens, B=B, L=L, keep=keep, first=rng.choice([0, 1, 4]),
                    recent=rng.choice([0, 16, keep // 4]), Hkv=Hkv, dqk=dqk, dv=dv, page=page)
    new = rng.choice(["one", "one", "mixed", "each"])
    L = _log(rng, 40, 24000 if wide else 48000)
    if new == "one":
        L = min(L, 400000 // B)
    else:
        L = min(L, 60000 // B + 40)
    chunk = 1 if new == "one" else min(L, _log(rng, 2, 1500 if new == "mixed" else max(3, 3000 // B)))
    return dict(op=op, lens=lens, B=B, L=L, new=new, chunk=chunk, window=rng.choice([0, 0, 0, 1000]), Hq=Hq, Hkv=Hkv,
                dqk=dqk, dv=dv, page=page)


def _split(case):
    """Tokens of each sequence, its new ones included: a function of the case alone."""
    L, n = case["L"], case["B"]
    if case["lens"] == "equal":
        return [L] * n
    low = max(1, min(L, 8))
    # spread over the logarithm, the longest first; odd lengths between
    return [max(1, int(round(L * (low / L) ** (i / max(1, n - 1)))) | (i & 1)) if i else L for i in range(n)]


def _new(case, lens):
    """New tokens of each sequence: one, a chunk each, or a chunk of the longest and one of all others."""
    if case["new"] == "mixed":
        return [min(case["chunk"], n) if i == 0 else 1 for i, n in enumerate(lens)]
    return [min(case["chunk"], n) for n in lens]


# ---------------------------------------------------------------- work

def _seen(n, m, window):
    """(pairs that m new tokens at the end of n see, cached tokens that one of them sees)."""
    first = n - m
    if not window:
        return sum(range(first + 1, n + 1)), n
    return sum(min(p + 1, window) for p in range(first, n)), min(n, m + window - 1)


def work(case):
    op, Hkv = case["op"], case["Hkv"]
    d = case["dqk"] + case["dv"]
    if op == "kv_write":
        n = case["T"] * Hkv * d
        return {"bytes": (4 if case["wide"] else 2) * n + 2 * n + 4 * case["T"] * (Hkv + 1), "flops": 0}
    lens = _split(case)
    if op == "kv_evict":
        kept = sum(min(n, case["keep"]) for n in lens) * Hkv
        return {"bytes": 4 * sum(lens) * Hkv + kept * (2 * (2 * d + 4) + 4), "flops": 0}
    new = _new(case, lens)
    pairs, tokens = (sum(x) for x in zip(*(_seen(n, m, case["window"]) for n, m in zip(lens, new))))
    T, Hq = sum(new), case["Hq"]
    if op == "kv_attn":
        return {"bytes": 2 * tokens * Hkv * d + T * Hq * (2 * d + 4), "flops": 2 * pairs * Hq * d}
    return {"bytes": 2 * tokens * Hkv * case["dqk"] + T * Hq * (2 * case["dqk"] + 4) + 4 * sum(lens) * Hkv,
            "flops": 2 * pairs * Hq * case["dqk"]}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    op, Hkv, page, dqk, dv = case["op"], case["Hkv"], case["page"], case["dqk"], case["dv"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    def heads(T, H, d, dtype=torch.bfloat16):
        """Values of a projection: channels differ in size, some sit off zero."""
        width = torch.exp(0.5 * normal(H, d))
        shift = normal(H, d) * (torch.rand((H, d), generator=gen, device=dev) < 0.1)
        return (0.5 * (normal(T, H, d) * width + 2 * shift)).to(dtype)

    def pool(pages, d):
        """Cached rows of a whole pool of pages."""
        width = torch.exp(0.5 * normal(Hkv, 1, d))
        shift = normal(Hkv, 1, d) * (torch.rand((Hkv, 1, d), generator=gen, device=dev) < 0.1)
        out = torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device=dev)
        step = max(1, 2 ** 26 // (Hkv * page * d))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            out[p:p + n] = 0.5 * (normal(n, Hkv, page, d) * width + 2 * shift)
        return out

    if op == "kv_write":
        T = case["T"]
        # runs of tokens start at pages of their own, as sequences' pages do
        runs = -(-T // case["run"])
        per = -(-case["run"] // page)
        pages = runs * per + 3
        first = torch.randperm(runs, generator=gen, device=dev) * per
        t = torch.arange(T, device=dev)
        slots = (first[t // case["run"]] * page + t % case["run"]).to(torch.int32)
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        dtype = torch.float32 if case["wide"] else torch.bfloat16
        s = dict(new=[heads(T, Hkv, dqk, dtype), heads(T, Hkv, dv, dtype)], slots=slots,
                 k=torch.zeros((pages, Hkv, page, dqk), dtype=torch.bfloat16, device=dev),
                 v=torch.zeros((pages, Hkv, page, dv), dtype=torch.bfloat16, device=dev),
                 weights=torch.rand((pages, Hkv, page), generator=gen, device=dev))
        return _with_cache(case, s)

    lens = _split(case)

    def tables(count, order):
        """A block table that deals the pages of `order` to sequences of the given lengths."""
        need = [-(-n // page) for n in count]
        table = torch.zeros((len(count), max(need)), dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        return table, at

    kv_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    if op == "kv_evict":
        left = [min(n, case["keep"]) for n in lens]
        pages = sum(-(-n // page) for n in lens) + sum(-(-n // page) for n in left) + 2
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table, used = tables(lens, order)
        out_table, _ = tables(left, order[used:])
        # a few tokens have most of the weight; some have none at all
        weights = torch.exp(2 * normal(pages, Hkv, page) - 3)
        weights[torch.rand(weights.shape, generator=gen, device=dev) < 0.05] = 0
        s = dict(k=pool(pages, dqk), v=pool(pages, dv), weights=weights, table=table, out_table=out_table,
                 lens=kv_lens, host_lens=lens)
        return _with_cache(case, s)

    new = _new(case, lens)
    pages = sum(-(-n // page) for n in lens) + 2
    table, _ = tables(lens, torch.randperm(pages, generator=gen, device=dev).to(torch.int32))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(k=pool(pages, dqk), v=pool(pages, dv), table=table, lens=kv_lens, host_lens=lens, cu=cu,
             cu_q=torch.tensor(cu, dtype=torch.int32, device=dev), q=heads(cu[-1], case["Hq"], dqk))
    if op == "kv_weights":
        # as the attention before has left it
        s["lse"] = _run_attn(dict(s, case=case), values=False)
        s["weights"] = torch.zeros((pages, Hkv, page), device=dev)
    return _with_cache(case, s)


def _with_cache(case, s):
    """The handle that a server keeps beside its pages."""
    s["case"] = case
    if own:
        import ring_attention_slope_gb300 as slope

        s["cache"] = slope.KVCache(s["k"].shape[0], case["page"], case["Hkv"], case["dqk"], case["dv"], k=s["k"],
                                   v=s["v"])
    return s


# ---------------------------------------------------------------- plain forms

def _run_write(s):
    if own:
        import ring_attention_slope_gb300 as slope

        slope.kv_write(s["cache"], *s["new"], s["slots"], weights=s["weights"])
        return s["k"], s["v"], s["weights"]
    n, page = s["case"]["T"] - s["case"]["pad"], s["case"]["page"]
    at = s["slots"][:n].long()
    for pool, rows in zip((s["k"], s["v"]), s["new"]):
        pool[at // page, :, at % page] = rows[:n].to(pool.dtype)
    s["weights"][at // page, :, at % page] = 0
    return s["k"], s["v"], s["weights"]


def _scores(s, b, heads):
    """Masked scores [heads, new * group, tokens] (fp32) of sequence b for a range of key heads, and its pages."""
    case, n = s["case"], s["host_lens"][b]
    group, m = case["Hq"] // case["Hkv"], s["cu"][b + 1] - s["cu"][b]
    pages = s["table"][b, :-(-n // case["page"])].long()
    k = s["k"][pages][:, heads].transpose(0, 1).flatten(1, 2)[:, :n].float()
    rows = s["q"][s["cu"][b]:s["cu"][b + 1]].float().unflatten(1, (-1, group))[:, heads]
    rows = rows.permute(1, 0, 2, 3).flatten(1, 2) / math.sqrt(case["dqk"])
    score = rows @ k.transpose(1, 2)
    key = torch.arange(n, device=k.device)
    pos = torch.arange(n - m, n, device=k.device)[:, None]
    hidden = key > pos
    if case["window"]:
        hidden |= pos - key >= case["window"]
    score.unflatten(1, (m, group)).masked_fill_(hidden[:, None], -math.inf)
    return score, pages


def _parts(s, b):
    """Ranges of key heads whose scores take up to 8 GB."""
    case = s["case"]
    each = (s["cu"][b + 1] - s["cu"][b]) * (case["Hq"] // case["Hkv"]) * s["host_lens"][b]
    step = max(1, 2 ** 31 // each)
    return [slice(h, min(case["Hkv"], h + step)) for h in range(0, case["Hkv"], step)]


def _run_attn(s, values=True):
    case = s["case"]
    T, Hkv, group = s["cu"][-1], case["Hkv"], case["Hq"] // case["Hkv"]
    if own and values:
        import ring_attention_slope_gb300 as slope

        how = dict(q_len=1) if case["new"] == "one" else dict(cu_q=s["cu_q"])
        return slope.kv_attn(s["q"], s["cache"], s["table"], s["lens"], window=case["window"], **how)
    out = torch.empty((T, Hkv, group, case["dv"]), dtype=torch.bfloat16, device=s["q"].device) if values else None
    lse = torch.empty((Hkv, group, T), device=s["q"].device)
    for b, n in enumerate(s["host_lens"]):
        at = slice(s["cu"][b], s["cu"][b + 1])
        for heads in _parts(s, b):
            score, pages = _scores(s, b, heads)
            top = score.amax(-1, keepdim=True)
            p = score.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            lse[heads, :, at] = (top + total.log()).squeeze(-1).unflatten(1, (-1, group)).transpose(1, 2)
            if values:
                v = s["v"][pages][:, heads].transpose(0, 1).flatten(1, 2)[:, :n].float()
                out[at, heads] = (p @ v / total).unflatten(1, (-1, group)).transpose(0, 1).to(out.dtype)
    lse = lse.flatten(0, 1)
    return (out.flatten(1, 2), lse) if values else lse


def _run_weights(s):
    case = s["case"]
    if own:
        import ring_attention_slope_gb300 as slope

        how = dict(q_len=1) if case["new"] == "one" else dict(cu_q=s["cu_q"])
        return slope.kv_attn_weights(s["q"], s["cache"], s["table"], s["lens"], s["lse"], s["weights"],
                                     window=case["window"], accumulate=False, **how)
    Hkv, page, group = case["Hkv"], case["page"], case["Hq"] // case["Hkv"]
    for b, n in enumerate(s["host_lens"]):
        lse = s["lse"].unflatten(0, (Hkv, group))[:, :, s["cu"][b]:s["cu"][b + 1]].transpose(1, 2).flatten(1, 2)
        token = torch.arange(n, device=lse.device)
        for heads in _parts(s, b):
            score, pages = _scores(s, b, heads)
            total = score.sub_(lse[heads, :, None]).exp_().sum(1)
            s["weights"][pages[token // page], heads, token % page] = total.t()
    return s["weights"]


def _choose(weights, case):
    """Positions [heads, keep] that stay, in order: of weights [heads, tokens], by size and then by position."""
    n, keep, recent = weights.shape[1], case["keep"], min(case["recent"], case["keep"])
    first = min(case["first"], keep - recent)
    token = torch.arange(n, device=weights.device)
    if n <= keep:
        return token.expand(weights.shape[0], n)
    w = weights.masked_fill((token < first) | (token >= n - recent), math.inf)
    return torch.sort(w, dim=1, descending=True, stable=True).indices[:, :keep].sort(1).values


def _run_evict(s):
    case, page = s["case"], s["case"]["page"]
    keep = case["keep"]
    if own:
        import ring_attention_slope_gb300 as slope

        kept, left = slope.kv_evict(s["cache"], s["weights"], s["table"], s["lens"], keep, first=case["first"],
                                    recent=case["recent"], out_table=s["out_table"])
        return kept, left, s["k"], s["v"], s["weights"]
    kept = torch.full((case["B"], case["Hkv"], keep), -1, dtype=torch.int32, device=s["k"].device)
    head = torch.arange(case["Hkv"], device=s["k"].device)[:, None]
    for b, n in enumerate(s["host_lens"]):
        token = torch.arange(n, device=s["k"].device)
        w = s["weights"][s["table"][b, token // page].long(), :, token % page].t()
        old = _choose(w, case)
        m = old.shape[1]
        kept[b, :, :m] = old
        src = s["table"][b].long()[old // page], head, old % page
        new = token[:m].expand_as(old)
        dst = s["out_table"][b].long()[new // page], head, new % page
        for pool in (s["k"], s["v"], s["weights"]):
            pool[dst] = pool[src]
    return kept, s["lens"].clamp(max=keep), s["k"], s["v"], s["weights"]


def run(state):
    return {"kv_write": _run_write, "kv_attn": _run_attn, "kv_weights": _run_weights,
            "kv_evict": _run_evict}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _dense(pool, row, n):
    """[heads, n, ...] of a sequence, page after page."""
    page = pool.shape[2]
    out = [pool[p, :, :min(page, n - i * page)] for i, p in enumerate(row[:-(-n // page)])]
    return torch.cat(out, 1)


def _exact_probabilities(s, b, rows, h):
    """Scaled scores of a sequence's new tokens `rows` and query head h over its keys, hidden ones -inf (64 bits)."""
    case, n = s["case"], s["host_lens"][b]
    g = h // (case["Hq"] // case["Hkv"])
    m = s["cu"][b + 1] - s["cu"][b]
    x = s["q"][s["cu"][b]:s["cu"][b + 1], h][rows].double() @ s["dense"][g].t() * case["dqk"] ** -0.5
    pos = torch.arange(m, device=x.device)[rows][:, None] + (n - m)
    gap = pos - torch.arange(n, device=x.device)
    seen = (gap >= 0) & (gap < case["window"]) if case["window"] else gap >= 0
    return torch.where(seen, x, -math.inf)


def exact(case, seed):
    op = case["op"]
    if op in ("kv_attn", "kv_weights"):
        lens = _split(case)
        pairs = sum(_seen(n, m, case["window"])[0] for n, m in zip(lens, _new(case, lens))) * case["Hq"]
        if pairs * (case["dqk"] + case["dv"]) > 3e12:
            return None  # over 20 seconds in 64 bits
    s = prepare(case, seed)
    page = case["page"]
    if op == "kv_write":
        pools = [s[x].double() for x in ("k", "v", "weights")]
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                for pool, rows in zip(pools, (*s["new"], None)):
                    pool[slot // page, :, slot % page] = 0 if rows is None else rows[t].double()
        return tuple(pools)
    table = s["table"].tolist()
    if op == "kv_evict":
        kept = torch.full((case["B"], case["Hkv"], case["keep"]), -1, dtype=torch.int64)
        pools = [s[x].double() for x in ("k", "v", "weights")]
        out_table = s["out_table"]
        for b, n in enumerate(s["host_lens"]):
            m, first, last = min(n, case["keep"]), case["first"], n - case["recent"]
            w = _dense(s["weights"], table[b], n).double().cpu().numpy()
            for h in range(case["Hkv"]):
                order = sorted(range(n), key=lambda t: (not (t < first or t >= last), -w[h, t], t)) if n > m else range(n)
                stay = torch.tensor(sorted(order[:m]))
                kept[b, h, :m] = stay
                new, old = torch.arange(m), stay.to(out_table.device)
                to, at = out_table[b].cpu().long()[new // page].to(old.device), (new % page).to(old.device)
                for pool, x in zip(pools, ("k", "v", "weights")):
                    pool[to, h, at] = _dense(s[x], table[b], n)[h].double()[old]
        return kept, torch.tensor([min(n, case["keep"]) for n in s["host_lens"]]), *pools
    dev, Hkv, group = s["q"].device, case["Hkv"], case["Hq"] // case["Hkv"]
    out = torch.zeros((s["cu"][-1], case["Hq"], case["dv"]), dtype=torch.float64, device=dev)
    lse = torch.zeros((case["Hq"], s["cu"][-1]), dtype=torch.float64, device=dev)
    weights = s["weights"].double() if op == "kv_weights" else None
    for b, n in enumerate(s["host_lens"]):
        s["dense"] = _dense(s["k"], table[b], n).double()
        v = _dense(s["v"], table[b], n).double()
        m = s["cu"][b + 1] - s["cu"][b]
        got = torch.zeros((Hkv, n), dtype=torch.float64, device=dev)
        for h in range(case["Hq"]):
            for r in range(0, m, 1024):
                rows = slice(r, min(m, r + 1024))
                at = slice(s["cu"][b] + rows.start, s["cu"][b] + rows.stop)
                x = _exact_probabilities(s, b, rows, h)
                if op == "kv_attn":
                    lse[h, at] = torch.logsumexp(x, -1)
                    out[at, h] = torch.exp(x - lse[h, at, None]) @ v[h // group]
                else:
                    got[h // group] += torch.exp(x - s["lse"][h, at, None].double()).sum(0)
        if op == "kv_weights":
            for t in range(0, n, page):
                weights[table[b][t // page], :, :min(page, n - t)] = got[:, t:t + page]
    return weights if op == "kv_weights" else (out, lse)
