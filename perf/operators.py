"""The feed-forward operators of libsvq as measured cases.

Four operators, each over matrices in the canonical SVQ form (18-bit codes,
a direction codebook, a radius table and a channel permutation per matrix):

* ``epilogue``: y = act(x What^T + bias) + residual, one matrix;
* ``glu``:      h = act(x Gate^T + bg) * (x Up^T + bu), two matrices;
* ``route``:    router scores of every token, its top experts and weights;
* ``moe``:      y = residual + sum_j weight_j Down_j (act(Gate_j x) * Up_j x),
  the experts of a token chosen by ids.

With ``own`` false the operators are computed in their plain form from the
canonical codes (decode in fp32, then products, sums and comparisons); with
``own`` true through the library's calls on its packed matrices.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the smallest call: one 512 x 1024 matrix, one token, everything in
        # the epilogue, fp32 out (a small head; latency is all that counts)
        dict(name="epi_512x1024_m1_f32", op="epilogue", n=512, k=1024, bd=8, m=1, act="gelu_tanh",
             bias=True, residual=True, out="f32"),
        # attention output projection of a 4B-class layer during decoding:
        # the residual stream is added where the product ends
        dict(name="epi_o_m1", op="epilogue", n=2560, k=4096, bd=7, m=1, act="none", bias=False,
             residual=True, out="bf16"),
        # a biased projection for a few sequences decoded together (ragged
        # batch of 7), odd row count, fp32 out
        dict(name="epi_1021x2560_m7_f32", op="epilogue", n=1021, k=2560, bd=6, m=7, act="none",
             bias=True, residual=False, out="f32"),
        # down projection over a 2048-token prompt, residual added
        dict(name="epi_down_m2048", op="epilogue", n=2560, k=9728, bd=7, m=2048, act="none",
             bias=False, residual=True, out="bf16"),
        # gate and up of a 4B-class layer, one decoded token
        dict(name="glu_m1", op="glu", n=9728, k=2560, bd=7, bd_up=8, m=1, act="silu", bias=False,
             out="bf16"),
        # the same for a batch of 13 sequences, with biases
        dict(name="glu_m13", op="glu", n=9728, k=2560, bd=6, bd_up=7, m=13, act="gelu_tanh",
             bias=True, out="bf16"),
        # the same over a 2048-token prompt
        dict(name="glu_m2048", op="glu", n=9728, k=2560, bd=7, bd_up=7, m=2048, act="silu",
             bias=False, out="bf16"),
        # router of a 128-expert layer, one decoded token
        dict(name="route_m1", op="route", m=1, experts=128, k=2048, topk=8, score="softmax",
             renorm=True, select_bias=False),
        # the same over a 512-token prompt, sigmoid scores with a selection bias
        dict(name="route_m512", op="route", m=512, experts=128, k=2048, topk=8, score="sigmoid",
             renorm=True, select_bias=True),
        # a whole 128-expert layer, one decoded token
        dict(name="moe_m1", op="moe", experts=128, n=768, k=2048, m=1, topk=8, act="silu",
             residual=True, out="bf16"),
        # the same for 7 sequences decoded together
        dict(name="moe_m7", op="moe", experts=128, n=768, k=2048, m=7, topk=8, act="silu",
             residual=False, out="bf16"),
        # the same over a 512-token prompt
        dict(name="moe_m512", op="moe", experts=128, n=768, k=2048, m=512, topk=8, act="silu",
             residual=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["epilogue", "glu", "route", "moe"])
    act = rng.choice(ACTS)
    flag = lambda: rng.random() < 0.5
    if op == "epilogue":
        m = _log(rng, 1, 2048)
        return dict(op=op, n=_log(rng, 33, 9728), k=8 * _log(rng, 16, 1216) if m <= 256 else 8 * _log(rng, 16, 320),
                    bd=rng.choice([6, 7, 8]), m=m, act=act, bias=flag(), residual=flag(),
                    out="f32" if m <= 16 and flag() else "bf16")
    if op == "glu":
        m = _log(rng, 1, 2048)
        return dict(op=op, n=_log(rng, 33, 9728), k=8 * _log(rng, 16, 320), bd=rng.choice([6, 7, 8]),
                    bd_up=rng.choice([6, 7, 8]), m=m, act=rng.choice(ACTS[1:]), bias=flag(),
                    out="f32" if m <= 16 and flag() else "bf16")
    if op == "route":
        e = rng.randint(8, 256)
        return dict(op=op, m=_log(rng, 1, 2048), experts=e, k=8 * _log(rng, 32, 320),
                    topk=rng.randint(1, min(e, 10)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=flag(), select_bias=flag())
    e = rng.randint(4, 128)
    return dict(op=op, experts=e, n=8 * rng.randint(12, 96), k=8 * rng.randint(32, 256),
                m=_log(rng, 1, 512), topk=rng.randint(1, min(e, 8)), act=rng.choice(ACTS[1:]),
                residual=flag(), out="bf16")


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(m, k, g):
    """N(0, 1), one channel in a hundred ten times larger, bf16."""
    x = torch.randn((m, k), generator=g, device="cuda")
    hot = torch.randperm(k, generator=g, device="cuda")[:max(1, k // 100)]
    x[:, hot] *= 10.0
    return x.to(torch.bfloat16)


def _matrices(count, n, k, bds, g):
    """``count`` canonical matrices: random codes, unit directions in the
    positive orthant, log-spaced radii, random permutations.  Tables are
    padded to 256 directions and 16 radii."""
    nbytes = (n * (k // 8) * 18 + 7) // 8
    bd = torch.tensor(bds, dtype=torch.int32, device="cuda")
    book = torch.randn((count, 256, 8), generator=g, device="cuda", dtype=torch.float64).abs()
    book = (book / book.norm(dim=2, keepdim=True)).to(torch.float16)
    row = torch.arange(256, device="cuda")
    book[row[None, :] >= (1 << bd)[:, None]] = 0
    steps = (1 << (10 - bd)).to(torch.float64)[:, None]
    j = torch.arange(16, device="cuda", dtype=torch.float64)[None, :]
    rad = 0.02 * math.sqrt(8.0) * 0.5 * torch.exp(j / (steps - 1) * math.log(8.0))
    rad = torch.where(j < steps, rad, torch.zeros_like(rad)).to(torch.float16)
    codes = torch.randint(0, 256, (count, nbytes), generator=g, device="cuda", dtype=torch.uint8)
    perm = torch.rand((count, k), generator=g, device="cuda").argsort(dim=1).to(torch.int32)
    return dict(n=n, k=k, bd=bd, codes=codes, book=book, rad=rad, perm=perm)


class _Canonical:
    """One matrix on the host, as the library's pack call takes it."""

    def __init__(self, n, k, bd, codes, book, rad, perm):
        self.n, self.k, self.bd, self.br = n, k, bd, 10 - bd
        self.codes = codes
        self.codebook = book[:1 << bd].view("uint16")
        self.radius = rad[:1 << (10 - bd)].view("uint16")
        self.perm = perm


def _packed(ms):
    """The matrices as the handles that a program keeps."""
    from bit_spherical_vector_amd import svq
    host = [ms[name].cpu().numpy() for name in ("bd", "codes", "book", "rad", "perm")]
    return [svq.pack(_Canonical(ms["n"], ms["k"], int(bd), codes, book, rad, perm))
            for bd, codes, book, rad, perm in zip(*host)]


def _inputs(case, seed):
    """Everything a program has before the call, on the GPU."""
    g = _gen(seed)
    op, m = case["op"], case["m"]
    s = dict(case)
    if op == "route":
        e, k = case["experts"], case["k"]
        s["x"] = _activations(m, k, g)
        s["w"] = (torch.randn((e, k), generator=g, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
        s["sb"] = 0.1 * torch.randn(e, generator=g, device="cuda") if case["select_bias"] else None
        return s
    n, k = case["n"], case["k"]
    s["x"] = _activations(m, k, g)
    if op == "epilogue":
        s["w"] = _matrices(1, n, k, [case["bd"]], g)
        s["b"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        s["r"] = torch.randn((m, n), generator=g, device="cuda").to(torch.bfloat16) if case["residual"] else None
    elif op == "glu":
        s["w"] = _matrices(1, n, k, [case["bd"]], g)
        s["w2"] = _matrices(1, n, k, [case["bd_up"]], g)
        s["b"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        s["b2"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
    else:
        e, topk = case["experts"], case["topk"]
        bds = [6 + i % 3 for i in range(e)]
        s["w"] = _matrices(e, n, k, bds, g)
        s["w2"] = _matrices(e, n, k, bds, g)
        s["w3"] = _matrices(e, k, n, bds, g)
        s["ids"] = torch.rand((m, e), generator=g, device="cuda").argsort(dim=1)[:, :topk].to(torch.int32).contiguous()
        s["wt"] = torch.softmax(torch.randn((m, topk), generator=g, device="cuda"), dim=1)
        s["r"] = torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16) if case["residual"] else None
    return s


def _out_type(case):
    return torch.float32 if case.get("out") == "f32" else torch.bfloat16


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from bit_spherical_vector_amd import svq
    op, m = case["op"], case["m"]
    if op == "route":
        s["ids"] = torch.empty((m, case["topk"]), dtype=torch.int32, device="cuda")
        s["wt"] = torch.empty((m, case["topk"]), dtype=torch.float32, device="cuda")
        s["call"] = svq.MoeRouteCall(s["x"], s["w"], s["ids"], s["wt"], score=case["score"],
                                     renormalize=case["renorm"], select_bias=s["sb"])
        return s
    s["y"] = torch.empty((m, case["k"] if op == "moe" else case["n"]), dtype=_out_type(case), device="cuda")
    packed = [_packed(s.pop(name)) for name in ("w", "w2", "w3") if name in s]
    if op == "epilogue":
        s["call"] = svq.EpilogueCall(packed[0][0], s["x"], s["y"], bias=s["b"], act=case["act"],
                                     residual=s["r"])
    elif op == "glu":
        s["call"] = svq.GluCall(packed[0][0], packed[1][0], s["x"], s["y"], act=case["act"],
                                bias_gate=s["b"], bias_up=s["b2"])
    else:
        s["call"] = svq.MoeFfnCall(packed[0], packed[1], packed[2], s["x"], s["ids"], s["wt"], s["y"],
                                   act=case["act"], residual=s["r"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _act(v, act):
    if act == "relu":
        return v.clamp_min(0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _fields(codes, count):
    """The 18-bit fields of each LSB-first stream (four fields in 9 bytes)."""
    e, nbytes = codes.shape
    pad = (-nbytes) % 9
    if pad:
        codes = torch.cat([codes, codes.new_zeros((e, pad))], dim=1)
    b = codes.view(e, -1, 9).to(torch.int32).unbind(2)
    f = torch.stack([b[0] | (b[1] << 8) | ((b[2] & 3) << 16),
                     (b[2] >> 2) | (b[3] << 6) | ((b[4] & 15) << 14),
                     (b[4] >> 4) | (b[5] << 4) | ((b[6] & 63) << 12),
                     (b[6] >> 6) | (b[7] << 2) | (b[8] << 10)], dim=2)
    return f.view(e, -1)[:, :count]


def _decoded(ms, pick=None):
    """fp32 weights [matrix, n, k] in permuted slot order, of all matrices or
    of those that ``pick`` names."""
    n, k = ms["n"], ms["k"]
    at = (lambda t: t) if pick is None else (lambda t: t.index_select(0, pick))
    bd = at(ms["bd"])[:, None]
    f = _fields(at(ms["codes"]), n * (k // 8))
    idx = f >> 8
    d = idx & ((1 << bd) - 1)
    r = idx >> bd
    e = f.shape[0]
    base = torch.arange(e, device=f.device)[:, None]
    w = at(ms["book"]).float().view(e * 256, 8)[base * 256 + d]
    w *= at(ms["rad"]).float().view(-1)[base * 16 + r][:, :, None]
    lane = torch.arange(8, dtype=torch.int32, device=f.device)
    w = torch.where(((f[:, :, None] >> lane) & 1).bool(), -w, w)
    return w.view(e, n, k)


def _dense(ms, x):
    """x What^T of one matrix, fp32: the slots take channels perm."""
    return x.float()[:, ms["perm"][0].long()] @ _decoded(ms)[0].T


def _plain_route(s):
    logits = s["x"].double() @ s["w"].double().T
    if s["score"] == "softmax":
        z = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
        p = z / z.sum(dim=1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logits))
    key = p if s["score"] == "sigmoid" else logits
    if s["sb"] is not None:
        key = p + s["sb"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    wt = p.gather(1, ids)
    if s["renorm"]:
        wt = wt / wt.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), wt.float()


def _plain_moe(s):
    m, topk, e = s["m"], s["topk"], s["experts"]
    x = s["x"].float()
    if m * topk <= 2 * e:
        # one product per slot with the slot's own matrices
        ids = s["ids"].view(-1).long()
        rows = x.repeat_interleave(topk, dim=0)
        take = lambda ms, v: torch.bmm(_decoded(ms, ids),
                                       v.gather(1, ms["perm"][ids].long())[:, :, None])[:, :, 0]
        h = _act(take(s["w"], rows), s["act"]) * take(s["w2"], rows)
        y = (take(s["w3"], h).view(m, topk, -1) * s["wt"][:, :, None]).sum(dim=1)
    else:
        # every token through every expert, kept by its weight there
        each = lambda ms, v: torch.bmm(v, _decoded(ms).transpose(1, 2))
        g = each(s["w"], x[:, s["w"]["perm"].long()].transpose(0, 1))
        u = each(s["w2"], x[:, s["w2"]["perm"].long()].transpose(0, 1))
        h = _act(g, s["act"]) * u
        d = each(s["w3"], h.gather(2, s["w3"]["perm"].long()[:, None, :].expand(-1, m, -1)))
        gate = torch.zeros((m, e), device=x.device).scatter_add_(1, s["ids"].long(), s["wt"])
        y = (d * gate.T[:, :, None]).sum(dim=0)
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(_out_type(s))


def run(s):
    if own:
        s["call"]()
        return (s["ids"], s["wt"]) if s["op"] == "route" else s["y"]
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "moe":
        return _plain_moe(s)
    y = _dense(s["w"], s["x"])
    if s["b"] is not None:
        y = y + s["b"]
    y = _act(y, s["act"])
    if s["op"] == "glu":
        u = _dense(s["w2"], s["x"])
        y = y * (u + s["b2"] if s["b2"] is not None else u)
    elif s["r"] is not None:
        y = y + s["r"].float()
    return y.to(_out_type(s))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _matrix_bytes(n, k, bd):
    """Codes, codebook, radii and a 16-bit permutation."""
    return n * k * 9 / 32 + (16 << bd) + (2 << (10 - bd)) + 2 * k


def work(case):
    m, k = case["m"], case["k"]
    esz = 4 if case.get("out") == "f32" else 2
    if case["op"] == "route":
        e = case["experts"]
        return dict(bytes=int(2 * m * k + 2 * e * k + 8 * m * case["topk"] + (4 * e if case["select_bias"] else 0)),
                    flops=int(2 * m * e * k))
    n = case["n"]
    if case["op"] == "epilogue":
        b = _matrix_bytes(n, k, case["bd"]) + 2 * m * k + esz * m * n
        b += (4 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        return dict(bytes=int(b), flops=int(2 * m * n * k))
    if case["op"] == "glu":
        b = _matrix_bytes(n, k, case["bd"]) + _matrix_bytes(n, k, case["bd_up"]) + 2 * m * k + esz * m * n
        return dict(bytes=int(b + (8 * n if case["bias"] else 0)), flops=int(4 * m * n * k))
    e, topk = case["experts"], case["topk"]
    hit = e * (1 - (1 - topk / e) ** m)  # experts that some token names, on average
    b = hit * (2 * _matrix_bytes(n, k, 7) + _matrix_bytes(k, n, 7))
    b += 2 * m * k + esz * m * k + 8 * m * topk + (2 * m * k if case["residual"] else 0)
    return dict(bytes=int(b), flops=int(6 * m * topk * n * k))


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_weight(ms, i):
    """Matrix i as What [n, k] in channel order, float64: code by code from
    the three bytes that hold it."""
    n, k = ms["n"], ms["k"]
    bd = int(ms["bd"][i])
    at = torch.arange(n * (k // 8), device=ms["codes"].device) * 18
    stream = torch.cat([ms["codes"][i].long(), ms["codes"].new_zeros(2).long()])
    byte = at // 8
    word = stream[byte] + 256 * stream[byte + 1] + 65536 * stream[byte + 2]
    code = (word >> (at % 8)) % (1 << 18)
    direction, radius = (code // 256) % (1 << bd), code // (256 << bd)
    length = ms["rad"][i].double()[radius]
    slots = torch.stack([length * ms["book"][i, :, l].double()[direction] * (1.0 - 2.0 * ((code // (1 << l)) % 2))
                         for l in range(8)], dim=1).view(n, k)
    w = torch.empty_like(slots)
    w[:, ms["perm"][i].long()] = slots
    return w


def exact(case, seed):
    s = _inputs(case, seed)
    x = s["x"].double()
    if case["op"] == "route":
        logits = (x[:, None, :] * s["w"].double()[None]).sum(dim=2) if s["m"] <= 64 else x @ s["w"].double().T
        p = torch.softmax(logits, dim=1) if case["score"] == "softmax" else torch.sigmoid(logits)
        ids, wt = [], []
        key = p + s["sb"].double() if s["sb"] is not None else p
        left = key.clone()
        for _ in range(case["topk"]):
            best = left.max(dim=1, keepdim=True).values
            first = (left == best).to(torch.int8).argmax(dim=1, keepdim=True)
            ids.append(first)
            wt.append(p.gather(1, first))
            left.scatter_(1, first, -math.inf)
        ids, wt = torch.cat(ids, dim=1), torch.cat(wt, dim=1)
        if case["renorm"]:
            wt = wt / wt.sum(dim=1, keepdim=True)
        return ids.to(torch.int32), wt
    if case["op"] == "moe":
        y = torch.zeros((case["m"], case["k"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            token, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
            if not len(token):
                continue
            g = _act(x[token] @ _exact_weight(s["w"], e).T, case["act"])
            h = g * (x[token] @ _exact_weight(s["w2"], e).T)
            y.index_add_(0, token, (h @ _exact_weight(s["w3"], e).T) * s["wt"][token, slot].double()[:, None])
        return y if s["r"] is None else y + s["r"].double()
    y = x @ _exact_weight(s["w"], 0).T
    if s["b"] is not None:
        y = y + s["b"].double()
    y = _act(y, case["act"])
    if case["op"] == "glu":
        u = x @ _exact_weight(s["w2"], 0).T
        return y * (u if s["b2"] is None else u + s["b2"].double())
    return y if s["r"] is None else y + s["r"].double()
