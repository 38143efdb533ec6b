"""Cases that measure the serving operators around the prefill attention, and their plain forms.

Four operators, in the order a serving process uses them:

* ``norm_rope``     RMS norm of every query and key head and the rotation by position, in one pass
* ``kv4_store``     keys and values quantised to 4 bits as they are written into a paged cache, and read back
* ``kv4_attn``      attention of the newest tokens of every sequence over that cache
* ``attn_varlen``   causal grouped attention over prompts of different lengths, packed one after another

``run`` computes a case with elementary torch operations, or, where ``own`` is true, with the calls of
``ring_attention_slope_gb300``.

The 4-bit format (see ``include/slope_serving.h``): a group of 32 consecutive channels of one token and head keeps
``min`` (bf16) and ``scale`` (bf16), and a channel is ``min + scale * code`` with a code in 0..15.  A cache is
``[page][head][16-token block]``, and a block holds the key codes, the value codes and the 32-bit words
``scale << 16 | min`` of its 16 tokens, in the order that the attention reads them.
"""
import math

import numpy as np
import torch

own = False

GROUP = 32   # channels that share one scale and minimum
BLOCK = 16   # tokens of a cache block
FIFTEENTH = float(np.float32(1.0 / 15.0))


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 16 sequences (64 query and 8 key/value heads of 64): launch latency
        dict(name="norm_rope_decode_16", op="norm_rope", T=16, Hq=64, Hkv=8, d=64, rot=64, begin=0, inter=False,
             scaled=False, far=32000),
        # a whole 32K prompt of the ring workload's heads
        dict(name="norm_rope_prompt_32k", op="norm_rope", T=32768, Hq=64, Hkv=8, d=64, rot=64, begin=0, inter=False,
             scaled=False, far=0),
        # an odd chunk at far positions, 192-wide heads that rotate only their last 64 channels, scaled for length
        dict(name="norm_rope_part_8191", op="norm_rope", T=8191, Hq=128, Hkv=128, d=192, rot=64, begin=128, inter=True,
             scaled=True, far=90000),
        # the new tokens of 32 decoding sequences, each into its own page
        dict(name="kv4_store_decode_32", op="kv4_store", T=32, Hkv=8, dqk=64, dv=64, page=64, run=1, pad=0),
        # one 12K prefill chunk into the cache's pages
        dict(name="kv4_store_chunk_12k", op="kv4_store", T=12288, Hkv=8, dqk=64, dv=64, page=64, run=64, pad=0),
        # a ragged batch of 192/128 heads with padding rows that have no slot
        dict(name="kv4_store_wide_5001", op="kv4_store", T=5001, Hkv=32, dqk=192, dv=128, page=16, run=16, pad=37),
        # one sequence of a thousand tokens: the smallest decode step
        dict(name="kv4_attn_1x1000", op="kv4_attn", lens="equal", B=1, L=1000, q_len=1, Hq=64, Hkv=8, dqk=64, dv=64,
             page=64, window=0),
        # a serving batch with contexts from a few tokens to 32K
        dict(name="kv4_attn_32x32k_ragged", op="kv4_attn", lens="ragged", B=32, L=32768, q_len=1, Hq=64, Hkv=8, dqk=64,
             dv=64, page=64, window=0),
        # eight long contexts
        dict(name="kv4_attn_8x100k", op="kv4_attn", lens="equal", B=8, L=102400, q_len=1, Hq=64, Hkv=8, dqk=64, dv=64,
             page=64, window=0),
        # four tokens at once (a drafted continuation) over wide heads, one query head for each key head
        dict(name="kv4_attn_wide_4x8k_q4", op="kv4_attn", lens="ragged", B=4, L=8192, q_len=4, Hq=32, Hkv=32, dqk=192,
             dv=128, page=16, window=0),
        # forty short prompts packed together
        dict(name="attn_varlen_40_short", op="attn_varlen", lens="short", n=40, T=2000, Hq=64, Hkv=8, dqk=64, dv=64,
             window=0),
        # a 12K token budget shared by five prompts
        dict(name="attn_varlen_5_in_12k", op="attn_varlen", lens="ragged", n=5, T=12288, Hq=64, Hkv=8, dqk=64, dv=64,
             window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "kv4_store", "kv4_attn", "kv4_attn", "attn_varlen"])
    wide = rng.random() < 0.4
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 5, 7, 8]) if wide else rng.choice([1, 4, 5, 7, 8, 8, 12])
    if op == "norm_rope":
        d = rng.choice([64, 128, 192])
        rot = 16 * rng.randint(1, d // 16)
        return dict(op=op, T=_log(rng, 1, 16000), Hq=Hkv * group, Hkv=Hkv, d=d, rot=rot,
                    begin=8 * rng.randint(0, (d - rot) // 8), inter=rng.random() < 0.5, scaled=rng.random() < 0.5,
                    far=rng.choice([0, 5000, 131072, 1 << 20]))
    dqk, dv = rng.choice([(128, 128), (192, 128), (128, 64), (64, 128)]) if wide else (64, 64)
    page = rng.choice([16, 32, 64, 128])
    if op == "kv4_store":
        T = _log(rng, 1, 12000)
        return dict(op=op, T=T, Hkv=Hkv, dqk=dqk, dv=dv, page=page, run=rng.choice([1, 5, page]),
                    pad=min(T - 1, rng.choice([0, 0, 3])))
    if op == "kv4_attn":
        B = _log(rng, 1, 64)
        L = _log(rng, 8, 24000 if wide else 48000)
        return dict(op=op, lens=rng.choice(["equal", "ragged"]), B=B, L=max(8, min(L, 400000 // B)),
                    q_len=rng.choice([1, 1, 1, 2, 5]), Hq=Hkv * group, Hkv=Hkv, dqk=dqk, dv=dv, page=page,
                    window=rng.choice([0, 0, 0, 1000]))
    n = _log(rng, 1, 60)
    return dict(op=op, lens=rng.choice(["short", "ragged"]), n=n, T=_log(rng, max(2 * n, 100), 6000 if wide else 9000),
                Hq=Hkv * group, Hkv=Hkv, dqk=dqk, dv=dv, window=rng.choice([0, 0, 0, 300]))


def _split(case):
    """Lengths of the sequences of a case: a function of the case alone."""
    if case["op"] == "kv4_attn":
        if case["lens"] == "equal":
            return [case["L"]] * case["B"]
        top, low, n = case["L"], max(1, min(case["L"], 8)), case["B"]
        # spread over the logarithm, the longest first; odd lengths between
        return [max(1, int(round(top * (low / top) ** (i / max(1, n - 1)))) | (i & 1)) if i else top for i in range(n)]
    n, T = case["n"], case["T"]
    weight = [1 + (7 * i) % 5 for i in range(n)] if case["lens"] == "short" else [0.6 ** min(i, 12) for i in range(n)]
    lens = [max(1, int(T * w / sum(weight))) for w in weight]
    lens[0] = max(1, lens[0] + T - sum(lens))
    return lens


# ---------------------------------------------------------------- work

def _pairs(lens, window):
    w = [min(n, window) if window else n for n in lens]
    return sum(m * (m + 1) // 2 + (n - m) * m for n, m in zip(lens, w))


def _row_bytes(d):
    """Bytes of one token's head of d channels in 4 bits: the codes and a word for each group."""
    return d // 2 + 4 * (d // GROUP)


def work(case):
    op = case["op"]
    if op == "norm_rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": 2 * n + 2 * n + 4 * case["T"], "flops": 5 * n}
    if op == "kv4_store":
        n = case["T"] * case["Hkv"]
        d = case["dqk"] + case["dv"]
        held = n * (_row_bytes(case["dqk"]) + _row_bytes(case["dv"]))
        # read the values, write the cache, read it again, write the values it stands for
        return {"bytes": 2 * n * d + 2 * held + 2 * n * d + 4 * case["T"], "flops": 6 * n * d}
    lens = _split(case)
    if op == "kv4_attn":
        q = case["q_len"]
        T = len(lens) * q
        seen = [min(n, case["window"] + q - 1) if case["window"] else n for n in lens]
        held = sum(seen) * case["Hkv"] * (_row_bytes(case["dqk"]) + _row_bytes(case["dv"]))
        io = T * case["Hq"] * (2 * case["dqk"] + 2 * case["dv"] + 4)
        return {"bytes": held + io, "flops": 2 * q * sum(seen) * case["Hq"] * (case["dqk"] + case["dv"])}
    T = sum(lens)
    io = 2 * T * ((case["Hq"] + case["Hkv"]) * (case["dqk"] + case["dv"])) + 4 * T * case["Hq"]
    return {"bytes": io, "flops": 2 * _pairs(lens, case["window"]) * case["Hq"] * (case["dqk"] + case["dv"])}


# ---------------------------------------------------------------- inputs

def _inv_freq(rot, scaled):
    """Rotation frequencies; `scaled` stretches the slow ones by 8 and ramps between slow and fast ones."""
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not scaled:
        return f, 1.0
    turns = [4096 * x / (2 * math.pi) for x in f]
    keep = [min(1.0, max(0.0, (t - 1.0) / 31.0)) for t in turns]
    return [x * k + x / 8 * (1 - k) for x, k in zip(f, keep)], 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def heads(T, H, d, size=0.5):
        """Values of a projection: channels differ in size, some sit off zero."""
        width = torch.exp(0.5 * normal(H, d))
        shift = normal(H, d) * (torch.rand((H, d), generator=gen, device=dev) < 0.1)
        return (size * (normal(T, H, d) * width + 2 * shift)).to(torch.bfloat16)

    op = case["op"]
    if op == "norm_rope":
        T, d = case["T"], case["d"]
        inv, factor = _inv_freq(case["rot"], case["scaled"])
        positions = torch.arange(T, device=dev, dtype=torch.int32)
        if case["far"]:
            positions = torch.randint(0, case["far"], (T,), generator=gen, device=dev, dtype=torch.int32)
        return dict(case=case, q=heads(T, case["Hq"], d, 2.0), k=heads(T, case["Hkv"], d, 2.0),
                    qw=1 + 0.1 * normal(d), kw=1 + 0.1 * normal(d), positions=positions, inv=inv, factor=factor,
                    freq=torch.tensor(inv, dtype=torch.float64, device=dev))
    if op == "kv4_store":
        T, page = case["T"], case["page"]
        # runs of tokens start at pages of their own, as sequences' pages do
        runs = -(-T // case["run"])
        per = -(-case["run"] // page)
        n_pages = runs * per + 3
        first = torch.randperm(runs, generator=gen, device=dev) * per
        t = torch.arange(T, device=dev)
        slots = (first[t // case["run"]] * page + t % case["run"]).to(torch.int32)
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        k, v = heads(T, case["Hkv"], case["dqk"]), heads(T, case["Hkv"], case["dv"])
        data = torch.zeros((n_pages, case["Hkv"], page // BLOCK, _block_bytes(case)), dtype=torch.uint8, device=dev)
        out = [torch.zeros_like(k), torch.zeros_like(v)]  # rows without a slot keep their zeros
        return dict(case=case, k=k, v=v, slots=slots, data=data, out=out)
    lens = _split(case)
    if op == "kv4_attn":
        page, B = case["page"], case["B"]
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + 2
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        table = torch.zeros((B, max(need)), dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        data = torch.empty((n_pages, case["Hkv"], page // BLOCK, _block_bytes(case)), dtype=torch.uint8, device=dev)
        step = max(1, 2 ** 27 // (page * case["Hkv"] * (case["dqk"] + case["dv"])))
        for p in range(0, n_pages, step):
            n = min(step, n_pages - p) * page
            k, v = heads(n, case["Hkv"], case["dqk"]), heads(n, case["Hkv"], case["dv"])
            data[p:p + n // page] = _pack(_quantise(k), _quantise(v), page)
        q = heads(B * case["q_len"], case["Hq"], case["dqk"])
        return dict(case=case, q=q, data=data, table=table,
                    lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    T = sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), torch.tensor(lens, device=dev))
    return dict(case=case, q=heads(T, case["Hq"], case["dqk"]), k=heads(T, case["Hkv"], case["dqk"]),
                v=heads(T, case["Hkv"], case["dv"]), cu=cu, seq=seq)


# ---------------------------------------------------------------- the 4-bit format in plain operations

def _block_bytes(case):
    return BLOCK * (_row_bytes(case["dqk"]) + _row_bytes(case["dv"]))


def _quantise(x):
    """codes [T, H, d] (uint8), and scale and min [T, H, d / 32] (bf16) of values [T, H, d]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low = g.amin(-1).to(torch.bfloat16)
    span = g.amax(-1) - low.float()
    scale = (span * FIFTEENTH).to(torch.bfloat16)
    scale = torch.where(scale.float() < 2.0 ** -126, torch.zeros_like(scale), scale)
    step = torch.where(scale == 0, torch.ones_like(scale), scale).double()
    # in 64 bits: a quotient next to a half has to fall on its own side
    code = ((g.double() - low.double()[..., None]) / step[..., None]).round().clamp(0, 15)
    code = torch.where((scale == 0)[..., None], torch.zeros_like(code), code)
    return code.to(torch.uint8).flatten(-2), scale, low


def _words(scale, low):
    """The 32-bit words as 4 bytes each, low byte first."""
    return torch.stack((low, scale), -1).view(torch.uint8)


def _pack(kq, vq, page):
    """Cache bytes [pages, H, page / 16, block] of whole pages of tokens."""
    (kc, ks, kl), (vc, vs, vl) = kq, vq
    n, H, dqk = kc.shape
    dv = vc.shape[2]
    P, nb, ng, nc = n // page, page // BLOCK, dqk // GROUP, dv // 64
    nib = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)  # noqa: E731
    # keys: lane (g, q) holds tokens g and g + 8, of each group the 8 channels from 8 q on
    k = nib(kc).view(P, nb, 2, 8, H, ng, 4, 4).permute(0, 4, 1, 3, 6, 2, 5, 7).reshape(P, H, nb, 8, 4, ng // 2, 16)
    k = k.permute(0, 1, 2, 5, 3, 4, 6).reshape(P, H, nb, -1)
    # values: lane (g, q) holds tokens 2 q, 2 q + 1, 2 q + 8, 2 q + 9, of each 64 channels the 4 from 4 g on in both groups
    v = nib(vc).view(P, nb, 2, 4, 2, H, nc, 2, 8, 2).permute(0, 5, 1, 6, 8, 3, 2, 4, 7, 9).reshape(P, H, nb, -1)
    w = torch.cat((_words(ks, kl), _words(vs, vl)), 2)  # [n, H, ngk + ngv, 4]
    w = w.view(P, nb, BLOCK, H, -1).permute(0, 3, 1, 2, 4).reshape(P, H, nb, -1)
    return torch.cat((k, v, w), -1)


def _unpack(data, dqk, dv):
    """Keys and values [..., H, tokens, d] (fp32) that cache pages [..., H, blocks, bytes] stand for."""
    lead = data.shape[:-1]
    ng, nc = dqk // GROUP, dv // 64
    nk, nv = BLOCK * dqk // 2, BLOCK * dv // 2
    m = len(lead)
    at = lambda order: list(range(m)) + [m + i for i in order]  # noqa: E731
    nib = lambda b: torch.stack((b & 15, b >> 4), -1).flatten(-2)  # noqa: E731
    k = data[..., :nk].reshape(*lead, ng // 2, 8, 4, 16).permute(at((1, 2, 0, 3))).reshape(*lead, 8, 4, 2, ng, 4)
    k = nib(k.permute(at((2, 0, 3, 1, 4))).reshape(*lead, BLOCK, dqk // 2))
    v = data[..., nk:nk + nv].reshape(*lead, nc, 8, 4, 2, 2, 2, 2)
    v = nib(v.permute(at((3, 2, 4, 0, 5, 1, 6))).reshape(*lead, BLOCK, dv // 2))
    w = data[..., nk + nv:].contiguous().view(torch.bfloat16).reshape(*lead, BLOCK, ng + 2 * nc, 2).float()

    def values(code, word):
        x = code.float().unflatten(-1, (-1, GROUP))
        return (x * word[..., 1:2] + word[..., 0:1]).flatten(-2).flatten(-3, -2)

    return values(k, w[..., :ng, :]), values(v, w[..., ng:, :])


# ---------------------------------------------------------------- plain forms

def _norm_rope(x, weight, cos, sin, case):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight
    a, r = case["begin"], case["rot"]
    part = y[..., a:a + r]
    if case["inter"]:
        u, w = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
    else:
        u, w = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
    return torch.cat((y[..., :a], turned, y[..., a + r:]), -1).to(x.dtype)


def _run_norm_rope(s):
    case = s["case"]
    if own:
        import ring_attention_slope_gb300 as slope

        rope = slope.Rope(s["inv"], begin=case["begin"], interleaved=case["inter"], attention_factor=s["factor"])
        return slope.qk_norm_rope(s["q"], s["k"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, rope=rope,
                                  positions=s["positions"])
    angle = s["positions"].double()[:, None, None] * s["freq"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    return _norm_rope(s["q"], s["qw"], cos, sin, case), _norm_rope(s["k"], s["kw"], cos, sin, case)


def _run_kv4_store(s):
    case, page = s["case"], s["case"]["page"]
    if own:
        import ring_attention_slope_gb300 as slope

        cache = slope.KV4Cache(s["data"].shape[0], page, case["Hkv"], case["dqk"], case["dv"], data=s["data"])
        slope.kv4_write(cache, s["k"], s["v"], s["slots"])
        return slope.kv4_read(cache, s["slots"], k_out=s["out"][0], v_out=s["out"][1])
    # the same cache kept as plain rows: codes two to a byte and words, one row for each slot
    n = case["T"] - case["pad"]
    at = s["slots"][:n].long()
    rows = s["data"].view(s["data"].shape[0] * page, -1)
    parts = []
    for x in (s["k"], s["v"]):
        code, scale, low = _quantise(x[:n])
        parts += [(code[..., 0::2] | (code[..., 1::2] << 4)).flatten(1), _words(scale, low).flatten(1)]
    rows[at] = torch.cat(parts, 1)
    held = rows[at].split([p.shape[1] for p in parts], 1)
    for out, code, word in ((s["out"][0], held[0], held[1]), (s["out"][1], held[2], held[3])):
        c = torch.stack((code & 15, code >> 4), -1).reshape(n, case["Hkv"], -1, GROUP).float()
        w = word.contiguous().view(torch.bfloat16).reshape(n, case["Hkv"], -1, 2).float()
        out[:n] = (c * w[..., 1:2] + w[..., 0:1]).flatten(-2).to(out.dtype)
    return tuple(s["out"])


def _softmax_attention(score, value):
    """Attention output and log-sum-exp of masked scores [..., rows, keys]; rows that see no key give 0 and -inf."""
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = p @ value / torch.where(total == 0, torch.ones_like(total), total)
    return out, (top + total.log()).squeeze(-1)


def _run_kv4_attn(s):
    case = s["case"]
    q, table, lens = s["q"], s["table"], s["lens"]
    B, n, Hkv, page = table.shape[0], case["q_len"], case["Hkv"], case["page"]
    if own:
        import ring_attention_slope_gb300 as slope

        cache = slope.KV4Cache(s["data"].shape[0], page, Hkv, case["dqk"], case["dv"], data=s["data"])
        return slope.kv4_attn(q, cache, table, lens, q_len=n, window=case["window"])
    group = case["Hq"] // Hkv
    k, v = _unpack(s["data"][table.long()], case["dqk"], case["dv"])  # [B, pages, Hkv, page, d]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))          # [B, Hkv, keys, d]
    rows = q.float().view(B, n, Hkv, group, -1).transpose(1, 2).flatten(2, 3) / math.sqrt(case["dqk"])
    score = rows @ k.transpose(-1, -2)
    key = torch.arange(k.shape[2], device=q.device)
    pos = (lens[:, None] - n + torch.arange(n, device=q.device))[..., None]  # [B, n, 1]
    hidden = key > pos
    if case["window"]:
        hidden |= pos - key >= case["window"]
    score.unflatten(2, (n, group)).masked_fill_(hidden[:, None, :, None], -math.inf)
    out, lse = _softmax_attention(score, v)
    out = out.unflatten(2, (n, group)).transpose(1, 2).reshape(B * n, case["Hq"], -1)
    lse = lse.unflatten(2, (n, group)).transpose(1, 2).reshape(B * n, case["Hq"])
    return out.to(q.dtype), lse.t().contiguous()


def _run_attn_varlen(s):
    case = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    if own:
        import ring_attention_slope_gb300 as slope

        return slope.attn_varlen(q, k, v, s["cu"], window=case["window"])
    T, Hkv, group = q.shape[0], case["Hkv"], case["Hq"] // case["Hkv"]
    k, v = (x.float().transpose(0, 1) for x in (k, v))                   # [Hkv, T, d]
    rows = q.float().view(T, Hkv, group, -1).permute(1, 2, 0, 3).flatten(1, 2) / math.sqrt(case["dqk"])
    score = rows @ k.transpose(-1, -2)                                    # [Hkv, group * T, T]
    row = torch.arange(T, device=q.device)
    hidden = (s["seq"][:, None] != s["seq"]) | (row > row[:, None])
    if case["window"]:
        hidden |= row[:, None] - row >= case["window"]
    score.unflatten(1, (group, T)).masked_fill_(hidden, -math.inf)
    out, lse = _softmax_attention(score, v)
    out = out.unflatten(1, (group, T)).permute(2, 0, 1, 3).reshape(T, case["Hq"], -1)
    return out.to(q.dtype), lse.view(case["Hq"], T)


def run(state):
    return {"norm_rope": _run_norm_rope, "kv4_store": _run_kv4_store, "kv4_attn": _run_kv4_attn,
            "attn_varlen": _run_attn_varlen}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rope(x, w, pos, inv, factor, case):
    y = x.double()
    y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
    out = y.clone()
    half = case["rot"] // 2
    for i, f in enumerate(inv):
        a = case["begin"] + (2 * i if case["inter"] else i)
        b = case["begin"] + (2 * i + 1 if case["inter"] else half + i)
        c, n = factor * torch.cos(pos.double() * f)[:, None], factor * torch.sin(pos.double() * f)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * n
        out[..., b] = y[..., b] * c + y[..., a] * n
    return out


def _exact_values(x):
    """What values [T, H, d] read back as, group by group."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[-1], GROUP):
        g = x[..., a:a + GROUP].double()
        low = g.min(-1, keepdim=True).values  # bf16 inputs: the minimum is a bf16 number
        scale = ((g.max(-1, keepdim=True).values - low).float() * FIFTEENTH).to(torch.bfloat16).double()
        code = torch.where(scale > 0, torch.round((g - low) / torch.where(scale > 0, scale, 1.0)), 0.0).clamp(0, 15)
        out[..., a:a + GROUP] = low + scale * code
    return out


def _exact_row(blocks, token, d, base, word0, value):
    """Channel-wise values [..., d] of one token of cache blocks [..., bytes], each byte found by its address."""
    cols = []
    for c in range(d):
        if value:
            g, j = (c % 32) // 4, c % 4 + 4 * (c % 64 // 32)
            lane, word = g * 4 + token % 8 // 2, (c // 64) * 128 + token % 2 + 2 * (token // 8)
            byte = base + (word // 128 * 32 + lane) * 16 + (word % 128) * 4 + j // 2
        else:
            q, j, w = c % 32 // 8, c % 8, token // 8 * (d // GROUP) + c // 32
            byte = base + (w // 4 * 32 + token % 8 * 4 + q) * 16 + w % 4 * 4 + j // 2
        cols.append((blocks[..., byte] >> (4 * (j % 2))) & 15)
    code = torch.stack(cols, -1).double()
    words = blocks[..., word0:word0 + 4 * (d // GROUP)].contiguous().view(torch.bfloat16).double()
    low, scale = words[..., 0::2], words[..., 1::2]
    return low.repeat_interleave(GROUP, -1) + scale.repeat_interleave(GROUP, -1) * code


def _exact_kv4_attn(s):
    case = s["case"]
    dqk, dv, n, page, Hkv = case["dqk"], case["dv"], case["q_len"], case["page"], case["Hkv"]
    group = case["Hq"] // Hkv
    nk, nv, words = BLOCK * dqk // 2, BLOCK * dv // 2, (dqk + dv) // GROUP
    outs, lses = [], []
    for b, L in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-L // page)].long()
        blocks = s["data"][pages].transpose(0, 1).flatten(1, 2)  # [Hkv, blocks, bytes]
        at = nk + nv
        k = torch.stack([_exact_row(blocks, t, dqk, 0, at + 4 * words * t, False) for t in range(BLOCK)], 2)
        v = torch.stack([_exact_row(blocks, t, dv, nk, at + 4 * (words * t + dqk // GROUP), True)
                         for t in range(BLOCK)], 2)
        k, v = k.flatten(1, 2)[:, :L], v.flatten(1, 2)[:, :L]
        for i in range(n):
            pos = L - n + i
            lo = max(0, pos - case["window"] + 1) if case["window"] else 0
            q = s["q"][b * n + i].double().view(Hkv, group, dqk)
            x = q @ k[:, lo:max(lo, pos + 1)].transpose(1, 2) / math.sqrt(dqk)
            lse = torch.logsumexp(x, -1)
            outs.append((torch.exp(x - lse[..., None]) @ v[:, lo:max(lo, pos + 1)]).flatten(0, 1))
            lses.append(lse.flatten())
    return torch.nan_to_num(torch.stack(outs), nan=0.0), torch.stack(lses, 1)


def _exact_attn_varlen(s):
    case = s["case"]
    group = case["Hq"] // case["Hkv"]
    out = torch.zeros((s["q"].shape[0], case["Hq"], case["dv"]), dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros((case["Hq"], s["q"].shape[0]), dtype=torch.float64, device=s["q"].device)
    for a, e in zip(s["cu"][:-1], s["cu"][1:]):
        i = torch.arange(e - a, device=out.device)
        gap = i[:, None] - i
        seen = (gap >= 0) & (gap < case["window"]) if case["window"] else gap >= 0
        for h in range(case["Hq"]):
            x = s["q"][a:e, h].double() @ s["k"][a:e, h // group].double().t() / math.sqrt(case["dqk"])
            x = torch.where(seen, x, -math.inf)
            lse[h, a:e] = torch.logsumexp(x, -1)
            out[a:e, h] = torch.exp(x - lse[h, a:e, None]) @ s["v"][a:e, h // group].double()
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return tuple(_exact_rope(s[x], s[w], s["positions"], s["inv"], s["factor"], case)
                     for x, w in (("q", "qw"), ("k", "kw")))
    if case["op"] == "kv4_store":
        n = case["T"] - case["pad"]
        k, v = _exact_values(s["k"]), _exact_values(s["v"])
        k[n:], v[n:] = 0, 0
        return k, v
    return _exact_kv4_attn(s) if case["op"] == "kv4_attn" else _exact_attn_varlen(s)
