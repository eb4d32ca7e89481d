"""The decode-step operators on 4-bit storage, as a user's program calls them,
with a plain form of each in elementary torch operations.

  lora    gptq_w4a16_lora: a packed INT4 projection with the low-rank adapters
          of many requests
  moe     gptq_w4a16_moe: a whole mixture-of-experts layer of packed experts
          for a few tokens, from the router's logits
  append  gptq_kv4_append: rotation of new queries and keys, and the new keys
          and values into a paged 4-bit cache
  attn    gptq_kv4_attention: attention over that cache

Sizes are those of the repository's workloads (4096, 11008, 14336, eight
experts of 14336 x 4096, groups of 32 .. 128) and generic ones.
"""
import math

import torch

own = False

DEV = "cuda:0" if torch.cuda.is_available() else "cpu"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one request, one token: a projection's latency
        dict(name="lora 1 token", op="lora", T=1, m=4096, d=4096, g=128, r=16, n=4, run=1,
             act=False),
        # a decode batch, every token another request, an act-order up-projection
        dict(name="lora 8 requests", op="lora", T=8, m=14336, d=4096, g=128, r=16, n=32, run=1,
             act=True),
        # requests with short prompts together, large rank, a down-projection
        dict(name="lora 93 tokens", op="lora", T=93, m=4096, d=11008, g=64, r=64, n=6, run=24,
             act=False),
        # one token of an eight-expert layer: two experts are read
        dict(name="moe 1 token", op="moe", T=1, E=8, k=2, d=4096, f=14336, g=128, act=False,
             masked=False, renorm=True),
        # a decode batch that reaches every expert
        dict(name="moe 24 tokens", op="moe", T=24, E=8, k=2, d=4096, f=14336, g=128, act=False,
             masked=False, renorm=True),
        # many small experts, act-order, some experts masked off for a token
        dict(name="moe 7 tokens of 32 experts", op="moe", T=7, E=32, k=4, d=2048, f=1408, g=64,
             act=True, masked=True, renorm=False),
        # the new token of each of 16 sequences
        dict(name="append 16 tokens", op="append", T=16, hq=32, hkv=8, D=128, rot=128,
             inter=False, page=16, g=128, f32=True),
        # a prompt, interleaved rotation of part of the head, fine groups
        dict(name="append a prompt of 4001", op="append", T=4001, hq=32, hkv=8, D=128, rot=64,
             inter=True, page=64, g=32, f32=False),
        # one short sequence: latency
        dict(name="attn 1 sequence", op="attn", B=1, hq=32, hkv=8, D=128, page=16, g=128, len=777,
             nq=1, window=0),
        # a ragged decode batch
        dict(name="attn 32 sequences", op="attn", B=32, hq=32, hkv=8, D=128, page=64, g=128,
             len=8000, nq=1, window=0),
        # two very long sequences, fine groups
        dict(name="attn 2 x 131000", op="attn", B=2, hq=32, hkv=8, D=128, page=128, g=64,
             len=131000, nq=1, window=0),
        # several drafted tokens a sequence, odd head count, sliding window
        dict(name="attn 9 drafts, window", op="attn", B=9, hq=21, hkv=3, D=64, page=32, g=32,
             len=5003, nq=5, window=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "moe", "append", "attn"])
    if op == "lora":
        d = 128 * _log(rng, 4, 112)
        return dict(op=op, T=_log(rng, 1, 200), m=_log(rng, 500, 14336), d=d,
                    g=rng.choice([64, 128, -1]), r=8 * _log(rng, 1, 12), n=_log(rng, 1, 40),
                    run=rng.choice([1, 1, 5, 30]), act=rng.random() < 0.5)
    if op == "moe":
        E = rng.choice([4, 8, 16, 33, 64])
        f = 128 * _log(rng, 4, max(8, 800 // E))
        return dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(E, 8)),
                    d=128 * _log(rng, 4, 32), f=f, g=rng.choice([32, 64, 128, -1]),
                    act=rng.random() < 0.3, masked=rng.random() < 0.3, renorm=rng.random() < 0.6)
    D = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 8])
    hq = hkv * rng.choice([1, 4, 7, 8, 12])
    g = rng.choice([x for x in (32, 64, 128) if D % x == 0] + [D])
    page = rng.choice([16, 32, 64, 256])
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 4001), hq=hq, hkv=hkv, D=D,
                    rot=rng.choice([D, D // 2, 32]), inter=rng.random() < 0.5, page=page, g=g,
                    f32=rng.random() < 0.5)
    B = _log(rng, 1, 48)
    length = _log(rng, 1, max(64, min(100000, 250000 // B)))
    return dict(op=op, B=B, hq=hq, hkv=hkv, D=D, page=page, g=g, len=length,
                nq=rng.choice([1, 1, 1, 2, 4, 9]), window=rng.choice([0, 0, 0, 500, 4000]))


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    return gen


def _activations(gen, n, d):
    """fp16 activations with 1 % of the channels as outliers"""
    x = torch.randn(n, d, generator=gen, device=DEV)
    x[:, torch.randperm(d, generator=gen, device=DEV)[: max(1, d // 100)]] *= 20.0
    return x.half()


def _packed(gen, lead, m, d, g, act):
    """A packed INT4 layer (or a stack): words, fp16 scales, zero nibbles, perm"""
    ng = 1 if g == -1 else d // g
    qw = torch.randint(-2 ** 31, 2 ** 31, (*lead, m, d // 8), generator=gen, device=DEV,
                       dtype=torch.int32)
    sc = (torch.rand(*lead, m, ng, generator=gen, device=DEV) * 0.006 + 0.004).half()
    qz = torch.randint(6, 10, (*lead, m, (ng + 1) // 2, 2), generator=gen, device=DEV,
                       dtype=torch.uint8)
    qz = qz[..., 0] | (qz[..., 1] << 4)
    perm = None
    if act:
        perm = torch.argsort(torch.rand(*lead, d, generator=gen, device=DEV), -1).int()
    return dict(qw=qw, sc=sc, qz=qz.contiguous(), perm=perm, g=g)


def _prepare_lora(c, gen):
    lay = _packed(gen, (), c["m"], c["d"], c["g"], c["act"])
    a = (torch.randn(c["n"], c["r"], c["d"], generator=gen, device=DEV) * 0.02).half()
    b = (torch.randn(c["n"], c["m"], c["r"], generator=gen, device=DEV) * 0.02).half()
    # consecutive tokens of one request share its adapter; -1: a request without one
    req = torch.arange(c["T"], device=DEV) // c["run"]
    ids = torch.randint(-1, c["n"], (c["T"],), generator=gen, device=DEV, dtype=torch.int32)
    scaling = torch.rand(c["n"], generator=gen, device=DEV) + 0.5
    return dict(x=_activations(gen, c["T"], c["d"]), lay=lay, a=a, b=b, ids=ids[req].contiguous(),
                scaling=scaling)


def _prepare_moe(c, gen):
    logits = torch.randn(c["T"], c["E"], generator=gen, device=DEV) * 2.0
    if c["masked"]:
        logits[torch.rand(c["T"], c["E"], generator=gen, device=DEV) < 0.25] = -math.inf
        logits[c["T"] // 2] = -math.inf         # a padding token: no expert at all
    return dict(x=_activations(gen, c["T"], c["d"]), logits=logits, k=c["k"], renorm=c["renorm"],
                inn=_packed(gen, (c["E"],), 2 * c["f"], c["d"], c["g"], c["act"]),
                out=_packed(gen, (c["E"],), c["d"], c["f"], c["g"], c["act"]))


def _table(n, rot):
    """cos | sin of every position (angles in 64 bits)"""
    inv = 500000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], -1).float().contiguous()


def _prepare_append(c, gen):
    T, hq, hkv, D, page = c["T"], c["hq"], c["hkv"], c["D"], c["page"]
    # the fused projection's output, of which q, k and v are views
    qkv = torch.randn(T, (hq + 2 * hkv) * D, generator=gen, device=DEV)
    qkv[:, torch.randperm(qkv.shape[1], generator=gen, device=DEV)[: qkv.shape[1] // 50]] *= 8.0
    qkv = qkv if c["f32"] else qkv.half()
    q = qkv[:, : hq * D].view(T, hq, D)
    k = qkv[:, hq * D: (hq + hkv) * D].view(T, hkv, D)
    v = qkv[:, (hq + hkv) * D:].view(T, hkv, D)
    decode = T <= 64                            # one token of each of T sequences, or one prompt
    pages = (T if decode else -(-T // page)) + 3
    order = torch.randperm(pages, generator=gen, device=DEV)
    j = torch.arange(T, device=DEV)
    if decode:
        slots = order[j] * page + torch.randint(0, page, (T,), generator=gen, device=DEV)
        pos = torch.randint(0, 8192, (T,), generator=gen, device=DEV)
    else:
        slots = order[j // page] * page + j % page
        pos = j + torch.randint(0, 8192 - T, (1,), generator=gen, device=DEV)
    cache = dict(kc=torch.zeros(pages, hkv, page, D // 8, dtype=torch.int32, device=DEV),
                 kp=torch.zeros(pages, hkv, page, D // c["g"], 2, dtype=torch.float16, device=DEV),
                 vc=torch.zeros(pages, hkv, page, D // 8, dtype=torch.int32, device=DEV),
                 vp=torch.zeros(pages, hkv, page, D // c["g"], 2, dtype=torch.float16, device=DEV))
    return dict(q=q, k=k, v=v, slots=slots, pos=pos.int(), table=_table(8192, c["rot"]),
                inter=c["inter"], cache=cache)


def _prepare_attn(c, gen):
    B, hkv, D, page = c["B"], c["hkv"], c["D"], c["page"]
    width = -(-c["len"] // page)
    lens = torch.randint(max(1, c["len"] // 4), c["len"] + 1, (B,), generator=gen, device=DEV)
    lens[0] = c["len"]
    if B > 4:
        lens[3] = 1                             # a sequence that just began
    nq = c["nq"] - torch.arange(B, device=DEV) % c["nq"]                  # ragged drafts
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), nq.cumsum(0)]).int()
    T = int(start[-1])
    pages = B * width + 1
    table = torch.randperm(pages, generator=gen, device=DEV)[: B * width].view(B, width)

    def half():
        codes = torch.randint(-2 ** 31, 2 ** 31, (pages, hkv, page, D // 8), generator=gen,
                              device=DEV, dtype=torch.int32)
        s = torch.rand(pages, hkv, page, D // c["g"], generator=gen, device=DEV) * 0.2 + 0.1
        z = torch.randint(6, 10, s.shape, generator=gen, device=DEV)
        return codes, torch.stack([s, z.float()], -1).half().contiguous()

    kc, kp = half()
    vc, vp = half()
    q = torch.randn(T, c["hq"], D, generator=gen, device=DEV).half()
    return dict(q=q, cache=dict(kc=kc, kp=kp, vc=vc, vp=vp), table=table.int().contiguous(),
                lens=lens.int(), start=start, scale=1.0 / math.sqrt(D), window=c["window"],
                max_nq=c["nq"], max_len=c["len"])


def prepare(case, seed):
    gen = _gen(seed)
    make = dict(lora=_prepare_lora, moe=_prepare_moe, append=_prepare_append, attn=_prepare_attn)
    return dict(make[case["op"]](case, gen), op=case["op"])


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _nibbles(words):
    """int32 words -> their eight nibbles each, along the last axis"""
    sh = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    return ((words[..., None] >> sh) & 15).flatten(-2)


def _weights(lay, pick=None):
    """The packed layer (or the picked ones of a stack) as fp32, in sweep order"""
    qw, sc, qz = (t if pick is None else t[pick] for t in (lay["qw"], lay["sc"], lay["qz"]))
    ng = sc.shape[-1]
    z = torch.stack([qz & 15, qz >> 4], -1).flatten(-2)[..., :ng]
    c = _nibbles(qw).float().unflatten(-1, (ng, -1))
    return ((c - z.float()[..., None]) * sc.float()[..., None]).flatten(-2)


def _plain_lora(s):
    x = s["x"].float()
    perm = s["lay"]["perm"]
    y = (x if perm is None else x[:, perm.long()]) @ _weights(s["lay"]).T
    ids = s["ids"].long()
    at = ids.clamp(min=0)
    t = torch.bmm(s["a"][at].float(), x[:, :, None])
    d = torch.bmm(s["b"][at].float(), t)[:, :, 0] * s["scaling"][at][:, None]
    return y + torch.where(ids[:, None] >= 0, d, torch.zeros_like(d))


def _plain_route(logits, k, renorm):
    l = torch.where(torch.isnan(logits), torch.full_like(logits, -math.inf), logits)
    top = l.amax(-1, keepdim=True)
    e = torch.where(l > -math.inf, torch.exp(l - top), torch.zeros_like(l))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    ids = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(-1, ids)
    if renorm:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return ids, w


def _plain_moe(s):
    x, T = s["x"].float(), s["x"].shape[0]
    E, d = s["out"]["qw"].shape[:2]
    ids, w = _plain_route(s["logits"], s["k"], s["renorm"])
    if ids.numel() < E:                         # the chosen experts, one for each token's choice
        pick = ids.flatten()
        xe = x.repeat_interleave(ids.shape[1], 0)[:, None]
        mix = None
    else:                                       # every expert on every token
        pick = torch.arange(E, device=x.device)
        xe = x[None].expand(E, -1, -1)
        mix = torch.zeros(T, E, device=x.device).scatter_add_(1, ids, w).T[:, :, None]

    def product(lay, v):
        if lay["perm"] is not None:
            at = lay["perm"][pick].long()
            v = v.gather(-1, at[:, None, :].expand(-1, v.shape[1], -1))
        return torch.bmm(v, _weights(lay, pick).transpose(1, 2))

    h = product(s["inn"], xe)
    gate, up = h.chunk(2, -1)
    out = product(s["out"], gate / (1 + torch.exp(-gate)) * up)
    if mix is not None:
        return (out * mix).sum(0)
    return (out[:, 0].unflatten(0, (T, -1)) * w[:, :, None]).sum(1)


def _plain_rotate(x, table, pos, inter):
    x = x.float()
    rot = table.shape[1]
    c, s = table[pos.long()][:, None].split(rot // 2, -1)
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else r.chunk(2, -1)
    p, q = a * c - b * s, b * c + a * s
    r = torch.stack([p, q], -1).flatten(-2) if inter else torch.cat([p, q], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_quantize(x, ng):
    """Asymmetric 4-bit groups: codes, fp16 scales, zero points (fp32 arithmetic)"""
    v = x.unflatten(-1, (ng, -1))
    lo = v.amin(-1).clamp(max=0)
    hi = v.amax(-1).clamp(min=0)
    flat = lo == hi
    lo, hi = torch.where(flat, -torch.ones_like(lo), lo), torch.where(flat, torch.ones_like(hi), hi)
    s = ((hi - lo) / 15).half().clamp(min=2.0 ** -24, max=65504.0)
    z = torch.round(-lo / s.float()).clamp(0, 15)
    c = (torch.round(v / s.float()[..., None]) + z[..., None]).clamp(0, 15)
    return c, s, z


def _key_order(c):
    """codes in head order -> the order of a key's words (and back: axes swapped)"""
    D = c.shape[-1]
    return c.unflatten(-1, (D // 32, 4, 8)).transpose(-3, -2).flatten(-3)


def _key_order_back(c):
    D = c.shape[-1]
    return c.unflatten(-1, (4, D // 32, 8)).transpose(-3, -2).flatten(-3)


def _value_order(c):
    D = c.shape[-1]
    return c.unflatten(-1, (D // 32, 8, 4)).transpose(-3, -2).flatten(-3)


def _value_order_back(c):
    D = c.shape[-1]
    return c.unflatten(-1, (8, D // 32, 4)).transpose(-3, -2).flatten(-3)


def _words(c):
    sh = torch.arange(0, 32, 4, device=c.device, dtype=torch.int64)
    w = (c.long().unflatten(-1, (-1, 8)) << sh).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def _plain_append(s):
    cache = s["cache"]
    ng, page = cache["kp"].shape[3], cache["kc"].shape[2]
    at = (s["slots"] // page, slice(None), s["slots"] % page)
    kr = _plain_rotate(s["k"], s["table"], s["pos"], s["inter"])
    held = []
    for x, codes, params, order in ((kr, cache["kc"], cache["kp"], _key_order),
                                    (s["v"].float(), cache["vc"], cache["vp"], _value_order)):
        c, sc, z = _plain_quantize(x, ng)
        codes[at] = _words(order(c.flatten(-2)))
        params[at] = torch.stack([sc, z.half()], -1)
        held.append(((c - z[..., None]) * sc.float()[..., None]).flatten(-2).half())
    q = _plain_rotate(s["q"], s["table"], s["pos"], s["inter"]).half()
    return [q, held[0], held[1], cache["kc"], cache["kp"], cache["vc"], cache["vp"]]


def _plain_attn(s):
    cache, q = s["cache"], s["q"].float()
    T, hq, D = q.shape
    B, width = s["table"].shape
    hkv, page = cache["kc"].shape[1:3]
    ng = cache["kp"].shape[3]

    def held(codes, params, back):              # [B, hkv, L, D]
        at = s["table"].long()
        c = back(_nibbles(codes[at])).float().unflatten(-1, (ng, -1))
        p = params[at].float()
        v = ((c - p[..., 1:]) * p[..., :1]).flatten(-2)
        return v.transpose(1, 2).flatten(2, 3)

    # queries of each sequence, padded to the longest
    n = s["max_nq"]
    start, lens = s["start"].long(), s["lens"].long()
    nq = start[1:] - start[:-1]
    i = torch.arange(n, device=q.device)
    row = (start[:-1, None] + i).clamp(max=T - 1)
    qp = q[row].unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    sc = torch.matmul(qp, held(cache["kc"], cache["kp"], _key_order_back).transpose(2, 3))
    sc = sc.unflatten(2, (-1, n)) * s["scale"]
    last = (lens - nq)[:, None] + i             # the last key that query i sees
    j = torch.arange(width * page, device=q.device)
    see = j <= last[..., None]
    if s["window"]:
        see = see & (j > last[..., None] - s["window"])
    sc = torch.where(see[:, None, None], sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(sc - top)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.flatten(2, 3), held(cache["vc"], cache["vp"], _value_order_back))
    o = o.unflatten(2, (-1, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)      # [B, n, hq, D]
    return o[i < nq[:, None]].half()


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _own(s):
    from post_weight_quantization_11_b200 import gptq as G
    if s["op"] == "lora":
        lay = s["lay"]
        return G.gptq_w4a16_lora(s["x"], lay["qw"], lay["sc"], lay["qz"], s["a"], s["b"], s["ids"],
                                 s["scaling"], group_size=lay["g"], perm=lay["perm"])
    if s["op"] == "moe":
        a, b = s["inn"], s["out"]
        return G.gptq_w4a16_moe(s["x"], s["logits"], a["qw"], a["sc"], a["qz"], b["qw"], b["sc"],
                                b["qz"], s["k"], group_size=a["g"], renormalize=s["renorm"],
                                perm_in=a["perm"], perm_out=b["perm"])
    c = s["cache"]
    cache = G.KV4Cache(c["kc"], c["kp"], c["vc"], c["vp"])
    if s["op"] == "append":
        q, k, v = G.gptq_kv4_append(s["k"], s["v"], s["pos"], s["slots"], s["table"], cache,
                                    q=s["q"], interleaved=s["inter"], values=True)
        return [q, k, v, c["kc"], c["kp"], c["vc"], c["vp"]]
    return G.gptq_kv4_attention(s["q"], cache, s["table"], s["lens"], s["start"], s["scale"],
                                window=s["window"], max_q_len=s["max_nq"],
                                max_seq_len=s["max_len"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "lora":
        return _plain_lora(state)
    if state["op"] == "moe":
        return _plain_moe(state)
    if state["op"] == "append":
        return _plain_append(state)
    return _plain_attn(state)


def work(case):
    c = case
    if c["op"] == "lora":
        ng = 1 if c["g"] == -1 else c["d"] // c["g"]
        layer = c["m"] * c["d"] / 2 + c["m"] * ng * 2.5
        requests = -(-c["T"] // c["run"])
        adapters = c["n"] * (1 - (1 - 1 / (c["n"] + 1)) ** requests)      # expected distinct
        ab = adapters * 2 * c["r"] * (c["d"] + c["m"])
        return {"bytes": layer + ab + 2 * c["T"] * c["d"] + 4 * c["T"] * c["m"],
                "flops": 2 * c["T"] * (c["m"] * c["d"] + c["r"] * (c["d"] + c["m"]))}
    if c["op"] == "moe":
        used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])             # expected distinct
        gd = c["d"] if c["g"] == -1 else c["g"]
        gf = c["f"] if c["g"] == -1 else c["g"]
        per = 2 * c["f"] * c["d"] * (0.5 + 2.5 / gd) + c["d"] * c["f"] * (0.5 + 2.5 / gf)
        return {"bytes": used * per + c["T"] * (6 * c["d"] + 4 * c["E"]),
                "flops": 6 * c["T"] * c["k"] * c["d"] * c["f"]}
    if c["op"] == "append":
        rows = c["T"] * (c["hq"] + 2 * c["hkv"]) * c["D"]
        held = c["T"] * 2 * c["hkv"] * (c["D"] / 2 + 4 * c["D"] / c["g"])
        return {"bytes": rows * (4 if c["f32"] else 2) + rows * 2 + held + c["T"] * 4 * c["rot"],
                "flops": rows * 6}
    seen = [c["len"]] + [c["len"] * 5 / 8] * (c["B"] - 1)                 # expected lengths
    seen = sum(min(x, c["window"] + c["nq"]) if c["window"] else x for x in seen)
    nq = (c["nq"] + 1) / 2
    return {"bytes": seen * c["hkv"] * (c["D"] + 8 * c["D"] / c["g"]) +
            c["B"] * nq * c["hq"] * c["D"] * 4,
            "flops": 4 * seen * nq * c["hq"] * c["D"]}


# --------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------

def _matrix64(lay, e=None):
    """Q in original column order, float64, of one packed layer"""
    words, sc, qz, perm = (None if t is None else (t if e is None else t[e])
                           for t in (lay["qw"], lay["sc"], lay["qz"], lay["perm"]))
    m, d = words.shape[0], words.shape[1] * 8
    code = torch.empty(m, d, dtype=torch.float64, device=words.device)
    for n in range(8):
        code[:, n::8] = torch.bitwise_and(words >> (4 * n), 15).double()
    g = d // sc.shape[1]
    q = torch.empty_like(code)
    for k in range(sc.shape[1]):
        z = torch.bitwise_and(qz[:, k // 2] >> (4 * (k % 2)), 15).double()
        q[:, k * g:(k + 1) * g] = sc[:, k].double()[:, None] * (code[:, k * g:(k + 1) * g] -
                                                                z[:, None])
    if perm is None:
        return q
    out = torch.empty_like(q)
    out[:, perm.long()] = q
    return out


def _exact_lora(s):
    x = s["x"].double()
    y = x @ _matrix64(s["lay"]).T
    for t, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            low = s["a"][a].double() @ x[t]
            y[t] += s["scaling"][a].double() * (s["b"][a].double() @ low)
    return y


def _exact_moe(s):
    x = s["x"].double()
    T, E = s["logits"].shape
    f = s["out"]["qw"].shape[2] * 8
    routes = [[] for _ in range(E)]
    for t, row in enumerate(s["logits"].double().tolist()):
        open_ = [e for e in range(E) if row[e] == row[e] and row[e] > -math.inf]
        chosen = sorted(open_, key=lambda e: (-row[e], e))[: s["k"]]
        if not chosen:
            continue
        top = row[chosen[0]]
        total = math.fsum(math.exp(row[e] - top) for e in (chosen if s["renorm"] else open_))
        for e in chosen:
            routes[e].append((t, math.exp(row[e] - top) / total))
    y = torch.zeros_like(x)
    for e in range(E):
        if not routes[e]:
            continue
        at = torch.tensor([t for t, _ in routes[e]], device=x.device)
        w = torch.tensor([w for _, w in routes[e]], device=x.device, dtype=torch.float64)
        v = x[at] @ _matrix64(s["inn"], e).T
        h = v[:, :f] * torch.sigmoid(v[:, :f]) * v[:, f:]
        y[at] += w[:, None] * (h @ _matrix64(s["out"], e).T)
    return y


def _exact_append(s):
    table, pos = s["table"].double(), s["pos"].long()
    half = table.shape[1] // 2
    cos, sin = table[pos, :half], table[pos, half:]

    def turned(x):
        x = x.double().clone()
        for i in range(half):
            u, v = (2 * i, 2 * i + 1) if s["inter"] else (i, i + half)
            a, b = x[..., u].clone(), x[..., v].clone()
            c, n = cos[:, i, None], sin[:, i, None]
            x[..., u] = a * c - b * n
            x[..., v] = a * n + b * c
        return x

    def stored(x):
        g = x.shape[-1] // s["cache"]["kp"].shape[3]
        out = torch.empty_like(x)
        for k in range(0, x.shape[-1], g):
            w = x[..., k:k + g]
            lo, hi = w.min(-1, keepdim=True).values, w.max(-1, keepdim=True).values
            lo, hi = torch.minimum(lo, 0 * lo), torch.maximum(hi, 0 * hi)
            lo, hi = torch.where(hi > lo, lo, lo - 1), torch.where(hi > lo, hi, hi + 1)
            sc = ((hi - lo) / 15).half().clamp(min=2.0 ** -24, max=65504.0).double()
            z = (-lo / sc).round().clamp(0, 15)
            out[..., k:k + g] = sc * (((w / sc).round() + z).clamp(0, 15) - z)
        return out

    return [turned(s["q"]), stored(turned(s["k"])), stored(s["v"].double()), None, None, None,
            None]


def _exact_attn(s):
    cache = s["cache"]
    hkv, page = cache["kc"].shape[1:3]
    T, hq, D = s["q"].shape
    nb, grp = D // 32, hq // hkv
    d = torch.arange(D, device=s["q"].device)
    knib = (((d % 32) // 8) * nb + d // 32) * 8 + d % 8            # nibble of d in a key's words
    vnib = (((d % 32) // 4) * nb + d // 32) * 4 + d % 4            # and in a value's
    out = torch.zeros(T, hq, D, dtype=torch.float64, device=s["q"].device)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    for b in range(len(lens)):
        n, L = start[b + 1] - start[b], lens[b]
        ids = s["table"][b, : -(-L // page)].long()
        for h in range(hkv):
            def rows(codes, params, nib):
                w = codes[ids, h].reshape(-1, D // 8)[:L]
                c = torch.bitwise_and(w[:, nib // 8] >> (4 * (nib % 8)).int(), 15).double()
                p = params[ids, h].reshape(-1, params.shape[3], 2)[:L].double()
                p = p.repeat_interleave(D // params.shape[3], 1)
                return (c - p[..., 1]) * p[..., 0]
            K, V = rows(cache["kc"], cache["kp"], knib), rows(cache["vc"], cache["vp"], vnib)
            for i in range(n):
                hi = L - n + i + 1
                lo = max(0, hi - s["window"]) if s["window"] else 0
                if hi <= lo:
                    continue
                q = s["q"][start[b] + i, h * grp:(h + 1) * grp].double()
                p = torch.softmax(s["scale"] * (q @ K[lo:hi].T), -1)
                out[start[b] + i, h * grp:(h + 1) * grp] = p @ V[lo:hi]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(lora=_exact_lora, moe=_exact_moe, append=_exact_append,
                attn=_exact_attn)[case["op"]](s)
