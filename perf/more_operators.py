"""The attention operators of libsvq as measured cases.

Four operators around a decoder layer's products:

* ``prompt``: attention of whole prompts, packed one behind another,
  y_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys that query i sees;
* ``write``:  keys and values of new tokens quantised into a paged cache of
  4-bit codes, and read back as the values it now holds;
* ``read``:   tokens of such a cache read back;
* ``cache``:  attention of the newest tokens over such a cache.

A group of channels of one token and head is stored as 4-bit codes c, a scale
s and a minimum m, both bf16, and stands for m + c * s: m is the group's
minimum, s = (maximum - minimum) / 15 rounded to fp32 and then to bf16, c the
nearest whole number to (x - m) / s (ties to even) within 0..15.

With ``own`` false the operators are computed in their plain form; with
``own`` true through the library's calls.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a 2048-token prompt of a 4B-class layer (32 query heads over 8 key
        # heads of 128 channels)
        dict(name="prompt_2048", op="prompt", lens="2048", heads=32, kv_heads=8, dim=128, causal=True, window=0,
             prefix=0),
        # prompts of several users in one batch, from one token to thousands,
        # a window of 1024 tokens, groups of 8 query heads
        dict(name="prompt_ragged_window", op="prompt", lens="1,17,130,333,64,1021,2,3001,777,255", heads=32,
             kv_heads=4, dim=128, causal=True, window=1024, prefix=0),
        # short texts through an encoder: every token sees its whole text,
        # one key head per query head, 64 channels
        dict(name="prompt_encode_64", op="prompt", lens="512,33,190,401,7,288,511,96,350,129,64,222", heads=16,
             kv_heads=16, dim=64, causal=False, window=0, prefix=0),
        # one long document
        dict(name="prompt_16384", op="prompt", lens="16384", heads=32, kv_heads=8, dim=128, causal=True, window=0,
             prefix=0),
        # one token of one sequence written while decoding, pages of 16
        dict(name="write_1", op="write", tokens=1, kv_heads=8, dim=128, group=64, page=16, out="f32"),
        # the keys and values of a 2048-token prompt
        dict(name="write_2048", op="write", tokens=2048, kv_heads=8, dim=128, group=64, page=64, out="f32"),
        # a stored prefix of 777 tokens taken out of the cache, 64 channels
        dict(name="read_777", op="read", tokens=777, kv_heads=16, dim=64, group=32, page=16, out="bf16"),
        # a long document's keys and values, read back for its next chunk
        dict(name="read_32768", op="read", tokens=32768, kv_heads=8, dim=128, group=64, page=64, out="bf16"),
        # one sequence of 777 tokens, the next token: latency is all
        dict(name="cache_b1_777", op="cache", lens="777", q_len=1, heads=32, kv_heads=8, dim=128, group=64, page=16,
             window=0),
        # one sequence of 32768 tokens
        dict(name="cache_b1_32768", op="cache", lens="32768", q_len=1, heads=32, kv_heads=8, dim=128, group=64,
             page=64, window=0),
        # five drafted tokens of each of 13 sequences checked at once, a
        # window, small groups
        dict(name="cache_b13_q5_window", op="cache", lens="9,130,4097,511,2048,1500,64,3333,17,1024,801,6,2999", q_len=5,
             heads=32, kv_heads=4, dim=128, group=32, page=32, window=2000),
        # 64 sequences decoded together, up to 8192 tokens each
        dict(name="cache_b64", op="cache", lens=",".join(str(8192 - 127 * i) for i in range(64)), q_len=1, heads=32,
             kv_heads=8, dim=128, group=64, page=64, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8, 16])
    return kv * rng.choice([1, 2, 4, 7, 8] if kv <= 4 else [1, 2, 4]), kv


def _text(values):
    return ",".join(str(v) for v in values)


def draw(rng):
    op = rng.choice(["prompt", "prompt", "write", "read", "cache", "cache"])
    heads, kv = _heads(rng)
    dim = rng.choice([64, 128, 128, 256])
    if op == "prompt":
        n = _log(rng, 1, 24)
        lens = [_log(rng, 1, max(2, 6000 // n)) for _ in range(n)]
        causal = rng.random() < 0.7
        window = _log(rng, 16, 2048) if causal and rng.random() < 0.4 else 0
        # a prefix that every sequence has in front of its new tokens
        prefix = _log(rng, 1, 1000) if rng.random() < 0.3 else 0
        return dict(op=op, lens=_text(lens), heads=heads, kv_heads=kv, dim=dim, causal=causal, window=window,
                    prefix=prefix)
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("write", "read"):
        return dict(op=op, tokens=_log(rng, 1, 4096), kv_heads=kv, dim=dim, group=group, page=page,
                    out=rng.choice(["f32", "bf16"]))
    batch = _log(rng, 1, 48)
    q_len = rng.choice([1, 1, 1, 2, 3, 8])
    lens = [q_len + _log(rng, 1, max(2, 100000 // batch)) for _ in range(batch)]
    return dict(op=op, lens=_text(lens), q_len=q_len, heads=heads, kv_heads=kv, dim=dim, group=group, page=page,
                window=_log(rng, 64, 4096) if rng.random() < 0.3 else 0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def _rows(n, heads, dim, g, offset=False):
    """bf16 rows of ``heads`` heads: N(0, 1); keys have some channels with a
    larger spread and an offset that all tokens share."""
    x = torch.randn((n, heads * dim), generator=g, device="cuda")
    if offset:
        hot = torch.randperm(heads * dim, generator=g, device="cuda")[:max(1, heads * dim // 32)]
        x[:, hot] = 2.0 * x[:, hot] + 4.0 * torch.randn(len(hot), generator=g, device="cuda")
    return x.to(torch.bfloat16)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _inputs(case, seed):
    g = _gen(seed)
    s = dict(case)
    kv, dim = case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        lens = _lens(case)
        s["lens_q"], s["lens_k"] = lens, [n + case["prefix"] for n in lens]
        s["q"] = _rows(sum(lens), case["heads"], dim, g)
        s["k"] = _rows(sum(s["lens_k"]), kv, dim, g, offset=True)
        s["v"] = _rows(sum(s["lens_k"]), kv, dim, g)
        return s
    page = case["page"]
    if case["op"] in ("write", "read"):
        n = case["tokens"]
        s["pages"] = (n + page - 1) // page + 3
        # the pages of one sequence, in the order in which they were free
        table = torch.randperm(s["pages"], generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        s["slots"] = (table[at // page] * page + at % page).to(torch.int32)
        s["k"] = _rows(n, kv, dim, g, offset=True)
        s["v"] = _rows(n, kv, dim, g)
        return s
    lens, q_len = _lens(case), case["q_len"]
    need = [(n + page - 1) // page for n in lens]
    s["pages"], width = sum(need) + 3, max(need)
    order = torch.randperm(s["pages"], generator=g, device="cuda")
    table = torch.zeros((len(lens), width), dtype=torch.int64, device="cuda")
    slots = []
    for b, (n, first) in enumerate(zip(lens, _starts(need))):
        table[b, :need[b]] = order[first:first + need[b]]
        at = torch.arange(n, device="cuda")
        slots.append(table[b, at // page] * page + at % page)
    s["all_slots"] = torch.cat(slots).to(torch.int32)
    s["table"] = table.to(torch.int32)
    s["lens_dev"] = _int32(lens)
    s["max_len"] = max(lens)
    s["q"] = _rows(len(lens) * q_len, case["heads"], dim, g)
    s["k"] = _rows(sum(lens), kv, dim, g, offset=True)
    s["v"] = _rows(sum(lens), kv, dim, g)
    return s


def _out_type(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def prepare(case, seed):
    s = _inputs(case, seed)
    op, kv, dim = case["op"], case["kv_heads"], case["dim"]
    s["scale"] = 1.0 / math.sqrt(dim)
    if op == "prompt":
        if own:
            from bit_spherical_vector_amd import svq
            s["y"] = torch.empty_like(s["q"])
            starts = _int32(_starts(s["lens_q"]))
            starts_k = _int32(_starts(s["lens_k"])) if case["prefix"] else None
            s["call"] = svq.AttnPromptCall(s["q"], s["k"], s["v"], s["y"], starts, head_dim=dim, starts_k=starts_k,
                                           causal=case["causal"], window=case["window"])
        return s
    if own:
        from bit_spherical_vector_amd import svq
        cache = svq.KvCache(s["pages"], case["page"], kv, dim, group=case["group"])
    else:
        cache = _PlainCache(s["pages"] * case["page"], kv, dim, case["group"])
    s["cache"] = cache
    if op in ("write", "read"):
        s["k_out"] = torch.empty(s["k"].shape, dtype=_out_type(case), device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        if own:
            s["write"] = svq.KvWriteCall(cache, s["k"], s["v"], s["slots"])
            s["read"] = svq.KvReadCall(cache, s["slots"], s["k_out"], s["v_out"])
            if op == "read":
                s["write"]()
        elif op == "read":
            cache.write(s["k"], s["v"], s["slots"])
        return s
    if own:
        svq.kv_write(cache, s["k"], s["v"], s["all_slots"])
        s["y"] = torch.empty_like(s["q"])
        s["call"] = svq.AttnCacheCall(cache, s["q"], s["y"], s["table"], s["lens_dev"], q_len=case["q_len"],
                                      max_len=s["max_len"], window=case["window"])
    else:
        cache.write(s["k"], s["v"], s["all_slots"])
    del s["k"], s["v"]
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

class _PlainCache:
    """Codes, one a byte, with their scales and minima, by slot."""

    def __init__(self, slots, heads, dim, group):
        self.shape = (heads, dim // group, group)
        side = lambda: dict(c=torch.zeros((slots, *self.shape), dtype=torch.uint8, device="cuda"),
                            s=torch.zeros((slots, *self.shape[:2]), dtype=torch.bfloat16, device="cuda"),
                            m=torch.zeros((slots, *self.shape[:2]), dtype=torch.bfloat16, device="cuda"))
        self.k, self.v = side(), side()

    def write(self, k, v, slots):
        at = slots.long()
        for side, x in ((self.k, k), (self.v, v)):
            x = x.view(len(at), *self.shape)
            lo, hi = x.amin(dim=3), x.amax(dim=3)
            s = ((hi.double() - lo.double()) / 15).float().to(torch.bfloat16)
            step = torch.where(s > 0, s, torch.ones_like(s)).double()[..., None]
            # values next to a border: 64 bits
            c = torch.round((x.double() - lo.double()[..., None]) / step).clamp_(0, 15)
            side["c"][at] = c.to(torch.uint8)
            side["s"][at] = s
            side["m"][at] = lo

    def values(self, side, at):
        """fp32 [tokens, heads, dim]."""
        x = side["c"][at].float() * side["s"][at].float()[..., None] + side["m"][at].float()[..., None]
        return x.view(len(at), self.shape[0], -1)

    def read(self, slots):
        at = slots.long()
        return self.values(self.k, at), self.values(self.v, at)


def _attend(q, k, v, scale, first, causal, window):
    """Queries q [heads, n, d] at positions first, first + 1, ... over keys k
    and values v [kv_heads, len, d]; fp32."""
    heads, n, d = q.shape
    kv, keys = k.shape[0], k.shape[1]
    out = torch.empty_like(q)
    per = heads // kv
    step = max(1, (1 << 27) // max(1, heads * keys))
    for at in range(0, n, step):
        part = q[:, at:at + step]
        m = part.shape[1]
        pos = first + at + torch.arange(m, device=q.device)
        # keys that some query of this part sees
        lo = max(0, first + at - window + 1) if window else 0
        hi = max(lo, min(keys, first + at + m)) if causal else keys
        score = part.reshape(kv, per * m, d) @ k[:, lo:hi].transpose(1, 2) * scale
        score = score.view(heads, m, hi - lo)
        if causal:
            j = torch.arange(lo, hi, device=q.device)
            seen = j[None, :] <= pos[:, None]
            if window:
                seen &= j[None, :] > pos[:, None] - window
            score = score.masked_fill(~seen, -math.inf)
        if hi == lo:
            out[:, at:at + m] = 0
            continue
        top = score.amax(dim=2, keepdim=True)
        p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(dim=2, keepdim=True)
        y = (p.view(kv, per * m, hi - lo) @ v[:, lo:hi]).view(heads, m, d)
        out[:, at:at + m] = y / torch.where(total == 0, torch.ones_like(total), total)
    return out


def _plain_prompt(s):
    dim, y = s["dim"], torch.empty_like(s["q"])
    split = lambda t, a, b: t[a:b].float().view(b - a, -1, dim).transpose(0, 1).contiguous()
    at_q, at_k = _starts(s["lens_q"]), _starts(s["lens_k"])
    for i, (n, keys) in enumerate(zip(s["lens_q"], s["lens_k"])):
        o = _attend(split(s["q"], at_q[i], at_q[i] + n), split(s["k"], at_k[i], at_k[i] + keys),
                    split(s["v"], at_k[i], at_k[i] + keys), s["scale"], keys - n, s["causal"], s["window"])
        y[at_q[i]:at_q[i] + n] = o.transpose(0, 1).reshape(n, -1).to(y.dtype)
    return y


def _plain_cache(s):
    y, dim, n = torch.empty_like(s["q"]), s["dim"], s["q_len"]
    lens = _lens(s)
    at = _starts(lens)
    for b, keys in enumerate(lens):
        # a window leaves the keys before it alone
        skip = max(0, keys - n - s["window"] + 1) if s["window"] else 0
        k, v = (t.transpose(0, 1).contiguous() for t in s["cache"].read(s["all_slots"][at[b] + skip:at[b] + keys]))
        q = s["q"][b * n:(b + 1) * n].float().view(n, -1, dim).transpose(0, 1).contiguous()
        o = _attend(q, k, v, s["scale"], keys - skip - n, True, s["window"])
        y[b * n:(b + 1) * n] = o.transpose(0, 1).reshape(n, -1).to(y.dtype)
    return y


def run(s):
    op = s["op"]
    if own:
        if op in ("write", "read"):
            if op == "write":
                s["write"]()
            s["read"]()
            return s["k_out"], s["v_out"]
        s["call"]()
        return s["y"]
    if op == "prompt":
        return _plain_prompt(s)
    if op == "cache":
        return _plain_cache(s)
    if op == "write":
        s["cache"].write(s["k"], s["v"], s["slots"])
    for out, x in zip((s["k_out"], s["v_out"]), s["cache"].read(s["slots"])):
        out.copy_(x.view(out.shape))
    return s["k_out"], s["v_out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _seen(n, keys, causal, window):
    """Pairs of query and visible key of one sequence."""
    if not causal:
        return n * keys
    total = 0
    first, last = keys - n, keys - 1  # positions of its queries
    if window:
        full = max(0, last - max(first, window - 1) + 1)  # queries whose window lies inside
        total += full * window
        last -= full
    return total + (last - first + 1) * (first + last + 2) // 2


def _token_bytes(case):
    """Codes, scales and minima of one token, keys and values."""
    return 2 * case["kv_heads"] * (case["dim"] // 2 + 4 * (case["dim"] // case["group"]))


def work(case):
    kv, dim = case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        lens, pre = _lens(case), case["prefix"]
        pairs = sum(_seen(n, n + pre, case["causal"], case["window"]) for n in lens)
        seen = [min(n + pre, case["window"] + n - 1) if case["window"] else n + pre for n in lens]
        return dict(bytes=4 * sum(lens) * case["heads"] * dim + 4 * sum(seen) * kv * dim,
                    flops=4 * pairs * case["heads"] * dim)
    if case["op"] in ("write", "read"):
        n, size = case["tokens"], 4 if case["out"] == "f32" else 2
        values = 2 * n * kv * dim
        b = n * _token_bytes(case) + size * values + 4 * n
        return dict(bytes=b + (2 * values if case["op"] == "write" else 0),
                    flops=(6 if case["op"] == "write" else 2) * values)
    lens, n = _lens(case), case["q_len"]
    pairs = sum(_seen(n, keys, True, case["window"]) for keys in lens)
    seen = sum(min(keys, case["window"] + n - 1) if case["window"] else keys for keys in lens)
    b = seen * _token_bytes(case) + 4 * len(lens) * n * case["heads"] * dim
    return dict(bytes=b, flops=4 * pairs * case["heads"] * dim)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _stored(x, group):
    """What the cache holds for rows x, float64 of the same shape."""
    g = x.double().reshape(x.shape[0], -1, group)
    low = g.min(dim=2, keepdim=True).values
    s = ((g.max(dim=2, keepdim=True).values - low) / 15).to(torch.float32).to(torch.bfloat16).double()
    t = torch.where(s > 0, (g - low) / s, torch.zeros_like(g))
    whole = torch.floor(t)
    rest = t - whole
    up = (rest > 0.5) | ((rest == 0.5) & (whole % 2 == 1))
    code = torch.clamp(whole + up, max=15)
    return (low + code * s).view(x.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    kv, dim, op = case["kv_heads"], case["dim"], case["op"]
    if op in ("write", "read"):
        return _stored(s["k"], case["group"]), _stored(s["v"], case["group"])
    if op == "prompt":
        lens_q, lens_k, causal = s["lens_q"], s["lens_k"], case["causal"]
        value = lambda t, rows: t[rows].double()
    else:
        lens_k = _lens(case)
        lens_q, causal = [case["q_len"]] * len(lens_k), True
        value = lambda t, rows: _stored(t[rows], case["group"])
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    per = case["heads"] // kv
    at_q, at_k = _starts(lens_q), _starts(lens_k)
    for b, (n, keys) in enumerate(zip(lens_q, lens_k)):
        rows = slice(at_k[b], at_k[b] + keys)
        k, v = value(s["k"], rows).view(keys, kv, dim), value(s["v"], rows).view(keys, kv, dim)
        q = s["q"][at_q[b]:at_q[b] + n].double().view(n, case["heads"], dim)
        o = y[at_q[b]:at_q[b] + n].view(n, case["heads"], dim)
        j = torch.arange(keys, device="cuda")
        for h in range(case["heads"]):
            kh, vh = k[:, h // per].T.contiguous(), v[:, h // per].contiguous()
            for a in range(0, n, 2048):
                logits = torch.mm(q[a:a + 2048, h], kh) / math.sqrt(dim)
                p = torch.arange(a, min(a + 2048, n), device="cuda")[:, None] + keys - n
                hidden = torch.zeros_like(logits, dtype=torch.bool)
                if causal:
                    hidden |= j > p
                if case["window"]:
                    hidden |= j <= p - case["window"]
                o[a:a + 2048, h] = torch.mm(torch.softmax(logits.masked_fill(hidden, -math.inf), dim=1), vh)
    return y
