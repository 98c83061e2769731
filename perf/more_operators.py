"""Measured cases of the key-value cache held in 4 bits: store, read, attend.

``store``   a step's tokens through the cache: per-head RMS norm of queries and
            keys (optional) and rotary positions, keys and values quantised as
            they are written to the page pool, and what was written read back.
``read``    the stored keys and values of whole requests, as 16-bit rows.
``attend``  causal attention of every request's new tokens (one in decode, a
            chunk in prefill) over its 4-bit keys and values.

A head's elements are quantised 32 at a time.  Of a group, m is the element
largest in magnitude (the positive one if both signs reach it), M is |m|
rounded up to five significant bits, with m's sign, and an element x becomes

    k = clamp(floor(8 x / M + 1/2), -7, 8),   which stands for   M k / 8,

a number that the 16-bit types hold exactly.  A token's row in a page is, for
every head, ceil(head_dim / 32) groups of 16 bytes with the codes k + 7, then
for every head and group M as a 16-bit number; a page holds as many such rows,
each rounded up to 16 bytes, as fit.

The plain forms are elementary torch operations in 32 bits, rounded once at
the end; where a code is chosen, next to a border between two of them, in 64.
``exact`` restates the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
LARGEST = {"f16": 31.0 * 2.0 ** 11, "bf16": 31.0 * 2.0 ** 123}     # of a group's M
FINEST = {"f16": 2.0 ** -21, "bf16": 2.0 ** -100}                 # M is a multiple of it


def _mha7b(**kw):
    """The 7B-shaped layer: 32 heads of 128, pages of 4096 16-bit elements: three tokens a page."""
    return dict(heads_q=32, heads_kv=32, head_dim=128, page_elems=4096, dtype="f16", **kw)


def _gqa13b(**kw):
    """A 13B-shaped layer (hidden size 5120, 40 heads) with 8 shared key heads: 17 tokens a page."""
    return dict(heads_q=40, heads_kv=8, head_dim=128, page_elems=5120, dtype="bf16", **kw)


def listed():
    return [
        # a single request's decode step, where latency counts
        dict(name="store_one", op="store", decode=1, ctx_lo=640, ctx_hi=640, chunks=0, new_lo=0, new_hi=0, chunk_ctx=0,
             norm=False, interleaved=False, rot=128, factor=1.0, **_mha7b()),
        # the serving trace's decode batch, whole-head rotary of the half layout
        dict(name="store_decode", op="store", decode=256, ctx_lo=8, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, norm=False, interleaved=False, rot=128, factor=1.0, **_mha7b()),
        # the prefill batch with normed heads, an interleaved rotary of half the
        # head, and positions stretched by four for a long context
        dict(name="store_prefill_norm", op="store", decode=0, ctx_lo=0, ctx_hi=0, chunks=32, new_lo=8, new_hi=512,
             chunk_ctx=8191, norm=True, interleaved=True, rot=64, factor=4.0, **_gqa13b()),
        # one request leaves the cache (for the host, or another cache)
        dict(name="read_one", op="read", decode=1, ctx_lo=640, ctx_hi=640, chunks=0, new_lo=0, new_hi=0, chunk_ctx=0,
             **_mha7b()),
        # long requests leave it together
        dict(name="read_gqa", op="read", decode=16, ctx_lo=17, ctx_hi=8192, chunks=0, new_lo=0, new_hi=0, chunk_ctx=0,
             **_gqa13b()),
        # one request, one token: the smallest attention call
        dict(name="decode_one", op="attend", decode=1, ctx_lo=640, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, softcap=0.0, **_mha7b()),
        # the trace's decode batch
        dict(name="decode_batch", op="attend", decode=256, ctx_lo=8, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, softcap=0.0, **_mha7b()),
        # shared key heads, contexts of very different lengths
        dict(name="decode_gqa", op="attend", decode=128, ctx_lo=17, ctx_hi=8192, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, softcap=0.0, **_gqa13b()),
        # one request with a very long context, scores capped: all of the GPU on one row
        dict(name="decode_long_capped", op="attend", decode=1, ctx_lo=131071, ctx_hi=131071, chunks=0, new_lo=0,
             new_hi=0, chunk_ctx=0, softcap=30.0, **_gqa13b()),
        # the prefill batch: 32 whole prompts
        dict(name="chunk_prefill", op="attend", decode=0, ctx_lo=0, ctx_hi=0, chunks=32, new_lo=8, new_hi=512,
             chunk_ctx=0, softcap=0.0, **_mha7b()),
        # a chunk of a long prompt over what earlier chunks stored
        dict(name="chunk_long", op="attend", decode=0, ctx_lo=0, ctx_hi=0, chunks=1, new_lo=1024, new_hi=1024,
             chunk_ctx=16383, softcap=0.0, **_gqa13b()),
        # the trace's mixed step: decode tokens and prompt chunks within 1024 tokens
        dict(name="step_mixed", op="attend", decode=200, ctx_lo=8, ctx_hi=640, chunks=4, new_lo=100, new_hi=312,
             chunk_ctx=0, softcap=0.0, **_mha7b()),
    ]


def _log(rng, lo, hi):
    """An odd whole number, spread over the logarithm of lo..hi."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))) | 1


def draw(rng):
    op = rng.choice(["store", "store", "read", "attend", "attend", "attend", "attend"])
    heads_kv, group = rng.choice([1, 2, 4, 5, 8, 8]), rng.choice([1, 2, 4, 5, 7, 8])
    if rng.random() < 0.3:
        heads_kv, group = rng.choice([20, 32, 40]), 1
    d = rng.choice([64, 80, 96, 128, 128, 128])
    per_page = rng.choice([1, 2, 4, 5, 16])
    while heads_kv * d * per_page > 8192:
        per_page = max(1, per_page // 2)
    c = dict(op=op, heads_q=heads_kv * group, heads_kv=heads_kv, head_dim=d, page_elems=heads_kv * d * per_page,
             dtype=rng.choice(["f16", "bf16"]))
    kind = "decode" if op == "read" else rng.choice(["decode", "decode", "chunk", "mixed"])
    # at most about 200 M cached elements a side (decode; a quarter of it to read back) and 10^10 scores times
    # heads (chunks)
    hi = _log(rng, 17, 32767)
    most = max(1, (50_000_000 if op == "read" else 200_000_000) // (heads_kv * d * hi))
    c["decode"] = _log(rng, 1, min(255, most)) if kind != "chunk" else 0
    c["ctx_lo"], c["ctx_hi"] = (rng.choice([0, 1, 7, hi // 2]), hi) if kind != "chunk" else (0, 0)
    c.update(chunks=0, new_lo=0, new_hi=0, chunk_ctx=0)
    if kind != "decode":
        new = _log(rng, 17, 1023)
        ctx = rng.choice([0, 0, _log(rng, 17, 8191)])
        c["chunks"] = _log(rng, 1, max(1, min(31, 4095 // new, int(4e9 / (new * (new + ctx) * c["heads_q"])))))
        c["new_lo"], c["new_hi"], c["chunk_ctx"] = rng.choice([1, new // 2, new]), new, ctx
        if kind == "mixed":  # the plain form pads every request to the longest
            c["ctx_hi"] = min(c["ctx_hi"], 1023)
            c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
            c["decode"] = min(c["decode"], 63)
    if op == "store":
        c.update(norm=rng.random() < 0.5, interleaved=rng.random() < 0.5, rot=rng.choice([d, d, 32]),
                 factor=rng.choice([1.0, 4.0]))
    if op == "attend":
        c["softcap"] = rng.choice([0.0, 0.0, 30.0])
    return c


# ---- what a case's sizes say: lengths are a fixed spread, the same for every seed ---------------


def _spread(n, lo, hi):
    """n whole numbers over lo..hi, evenly spread in a scrambled order."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.5) % 1.0)) for i in range(n)]


def _lengths(c):
    """(tokens already stored, new tokens) of every request of the batch."""
    ctx = _spread(c["decode"], c["ctx_lo"], c["ctx_hi"]) + [c["chunk_ctx"]] * c["chunks"]
    new = [1] * c["decode"] + _spread(c["chunks"], c["new_lo"], c["new_hi"])
    return ctx, new


def _page(c):
    """(groups of a head, bytes of a token's row, tokens a page holds)."""
    ng = -(-c["head_dim"] // 32)
    rb = -(-18 * ng * c["heads_kv"] // 16) * 16
    return ng, rb, 2 * c["page_elems"] // rb


def work(c):
    ctx, new = _lengths(c)
    T, R = sum(new), len(new)
    d, hq, hkv = c["head_dim"], c["heads_q"], c["heads_kv"]
    ng, _, P = _page(c)
    held = 2 * 18 * ng * hkv                   # bytes of a token's keys and values
    lens = [a + n for a, n in zip(ctx, new)]
    if c["op"] == "store":
        return {"bytes": T * (4 * d * hq + 8 * d * hkv + 2 * held + 12), "flops": T * (10 * d * hq + 24 * d * hkv)}
    if c["op"] == "read":
        return {"bytes": sum(lens) * (held + 4 * d * hkv + 8), "flops": 4 * sum(lens) * d * hkv}
    scores = sum(n * a + n * (n + 1) // 2 for a, n in zip(ctx, new))
    return {"bytes": 4 * T * hq * d + sum(lens) * held + sum(8 * -(-n // P) for n in lens), "flops": 4 * d * hq * scores}


# ---- the format ---------------------------------------------------------------------------------


def _places(ng, values):
    """Where each element's code lies among a head's 4-bit places (low half of a byte first)."""
    e = torch.arange(32 * ng, device=DEV)
    g, r = e // 32, e % 32
    if values:
        return ((r // 4) * ng + g) * 4 + r % 4
    return ((r // 8) * ng + g) * 8 + (r % 8) // 2 + 4 * (r % 2)


def _quantise(x, dtype, ng):
    """x [..., heads, d] in 64 bits: codes [..., heads, 32 ng] (uint8) and M [..., heads, ng]."""
    d = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, 32 * ng - d)).unflatten(-1, (ng, 32))
    hi, lo = x.amax(-1), x.amin(-1)
    m = torch.where(hi >= -lo, hi, lo)
    ex = torch.frexp(m.abs()).exponent
    unit = ((ex.long() + (1023 - 5)) << 52).view(torch.float64).clamp(min=FINEST[dtype])   # 2^(ex - 5)
    M = torch.copysign(torch.ceil(m.abs() / unit) * unit, m).clamp(-LARGEST[dtype], LARGEST[dtype])
    k = torch.floor(8.0 * x / torch.where(M == 0, 1.0, M)[..., None] + 0.5).clamp(-7, 8)
    return (k + 7).to(torch.uint8).flatten(-2), M


def _rows(codes, M, tdt, rb, values):
    """Token rows [N, rb] (bytes) of codes [N, heads, 32 ng] and M [N, heads, ng]."""
    N, heads, ng = M.shape
    nibbles = torch.empty_like(codes)
    nibbles[..., _places(ng, values)] = codes
    rows = torch.zeros((N, rb), dtype=torch.uint8, device=DEV)
    rows[:, : heads * 16 * ng] = (nibbles[..., 0::2] | nibbles[..., 1::2] << 4).reshape(N, -1)
    rows[:, heads * 16 * ng: heads * 18 * ng] = M.to(tdt).reshape(N, -1).view(torch.uint8)
    return rows


def _values(rows, heads, d, tdt, values):
    """What rows [..., rb] stand for: [..., heads, d] in 32 bits."""
    ng, lead = -(-d // 32), rows.shape[:-1]
    b = rows[..., : heads * 16 * ng].reshape(*lead, heads, 16 * ng)
    nibbles = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    k = nibbles[..., _places(ng, values)[:d]].float() - 7.0
    M = rows[..., heads * 16 * ng: heads * 18 * ng].contiguous().view(tdt).view(*lead, heads, ng).float()
    return M.repeat_interleave(32, -1)[..., :d] * k * 0.125


def _row_view(s):
    """The pool as [page, token of the page, byte of its row]."""
    page_bytes = 2 * s["case"]["page_elems"]
    return s["buf"].view(torch.uint8).as_strided((s["num_pages"], s["P"], s["rb"]), (page_bytes, s["rb"], 1))


# ---- inputs -------------------------------------------------------------------------------------


def _inv_freq(c):
    """Rotary frequencies (radians a position) in 64 bits, positions stretched by `factor`."""
    return [10000.0 ** (-2.0 * i / c["rot"]) / c["factor"] for i in range(c["rot"] // 2)]


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    tdt = torch.float16 if c["dtype"] == "f16" else torch.bfloat16
    hq, hkv, d, H = c["heads_q"], c["heads_kv"], c["head_dim"], c["page_elems"]
    ng, rb, P = _page(c)
    ctx, new = _lengths(c)
    R, T = len(new), sum(new)
    i32 = dict(dtype=torch.int32, device=DEV)
    first = torch.tensor([-(-a // P) for a in ctx], device=DEV)            # blocks stored before the step
    total = torch.tensor([-(-(a + n) // P) for a, n in zip(ctx, new)], device=DEV)
    max_blocks, max_rows = max(1, int(total.max())), R + 3
    req = torch.repeat_interleave(torch.arange(R, device=DEV), total)
    blk = torch.arange(req.numel(), device=DEV) - (torch.cumsum(total, 0) - total)[req]
    fresh = blk >= first[req]
    # store writes the new tokens' blocks, the others read every block: the pool holds the
    # blocks whose contents count, the table names any page for the rest
    held = torch.ones_like(fresh) if c["op"] != "store" else (blk >= torch.tensor([a // P for a in ctx], device=DEV)[req])
    n_held = int(held.sum())
    num_pages = n_held * 2 + 5
    s = dict(case=c, P=P, rb=rb, ng=ng, R=R, T=T, num_pages=num_pages, max_blocks=max_blocks, max_new=max(new), tdt=tdt)
    s["rows"] = torch.randperm(max_rows, generator=g, device=DEV)[:R].to(torch.int32)   # table row of each request
    s["ctx"], s["new"] = torch.tensor(ctx, **i32), torch.tensor(new, **i32)
    pages = torch.randint(num_pages, (req.numel(), 2), generator=g, **i32)              # in no order: [block][K, V]
    pages[held] = torch.randperm(num_pages, generator=g, device=DEV)[: n_held * 2].to(torch.int32).view(-1, 2)
    s["pages"] = pages[fresh].reshape(-1).contiguous()                     # what the step's allocation handed out
    table = torch.full((1, 2, max_rows, max_blocks), -1, **i32)
    table[0, :, s["rows"].long()[req], blk] = pages.T
    s["table"] = table
    s["buf"] = torch.zeros((num_pages, H), dtype=tdt, device=DEV)
    view = _row_view(s)
    if c["op"] != "store":
        step = max(1, (1 << 25) // (P * hkv * d))
        for j in (0, 1):
            for at in range(0, n_held, step):
                to = pages[held][at: at + step, j].long()
                x = torch.empty((to.numel() * P, hkv, d), dtype=tdt, device=DEV).normal_(generator=g)
                view[to] = _rows(*_quantise(x.double(), c["dtype"], ng), tdt, rb, j == 1).view(-1, P, rb)
    if c["op"] == "store":
        qkv = torch.empty((T, (hq + 2 * hkv) * d), dtype=tdt, device=DEV).normal_(generator=g)   # one fused product's rows
        s["q"], s["k"], s["v"] = qkv[:, : hq * d], qkv[:, hq * d: (hq + hkv) * d], qkv[:, (hq + hkv) * d:]
        s["q_out"] = torch.empty((T, hq * d), dtype=tdt, device=DEV)
        s["qw"] = s["kw"] = None
        if c["norm"]:
            w = torch.empty((2, d), device=DEV).normal_(generator=g) * 0.2 + 1.0
            s["qw"], s["kw"] = w.to(tdt).unbind(0)
        s["inv_freq"] = _inv_freq(c)
        s["inv_freq64"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=DEV)
    if c["op"] == "attend":
        s["q"] = torch.empty((T, hq * d), dtype=tdt, device=DEV).normal_(generator=g) * 2.0
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(d)
    else:                                                                  # what is read back: (table row, position)
        lens = s["ctx"].long() + s["new"].long() if c["op"] == "read" else s["new"].long()
        r = torch.repeat_interleave(torch.arange(R, device=DEV), lens)
        p = torch.arange(r.numel(), device=DEV) - (torch.cumsum(lens, 0) - lens)[r]
        s["at_row"] = s["rows"][r].contiguous()
        s["at_pos"] = (p if c["op"] == "read" else p + s["ctx"].long()[r]).to(torch.int32)
        s["k_read"], s["v_read"] = (torch.empty((r.numel(), hkv * d), dtype=tdt, device=DEV) for _ in "kv")
    if own:
        from lora_adapters_gb300 import slora

        pool = slora.Pool(num_pages, H, c["dtype"], [(8, 8)], 1, 1, T, device=torch.device(DEV, torch.cuda.current_device()),
                          buffer=s["buf"])
        kv = slora.KVCache(pool, 1, hq, hkv, d, max_rows, max_blocks, bits=4)
        kv.table.copy_(table)
        s["pool"], s["kv"] = pool, kv
        if c["op"] == "store":
            kv.set_rotary(c["rot"], s["inv_freq"], interleaved=c["interleaved"])
        s["batch"] = kv.plan(s["ctx"], s["new"], s["pages"], T, s["max_new"], rows=s["rows"])
    return s


# ---- plain forms --------------------------------------------------------------------------------


def _positions(s):
    """(request, position) of every new token."""
    new, ctx = s["new"].long(), s["ctx"].long()
    ends = torch.cumsum(new, 0)
    tok = torch.arange(s["T"], device=DEV)
    req = torch.searchsorted(ends, tok, right=True)
    return req, ctx[req] + tok - (ends - new)[req]


def _rotate(x, s, pos):
    """The rotary turn of x [T, heads, d], in x's precision; angles in 64 bits."""
    c = s["case"]
    rot = c["rot"]
    ang = pos.double()[:, None] * s["inv_freq64"]
    cos, sin = torch.cos(ang).to(x.dtype)[:, None], torch.sin(ang).to(x.dtype)[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., : rot // 2], x[..., rot // 2: rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], -1).flatten(-2) if c["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_read(s):
    c, P = s["case"], s["P"]
    d, hkv, view = c["head_dim"], c["heads_kv"], _row_view(s)
    row, pos = s["at_row"].long(), s["at_pos"].long()
    out = []
    for j in (0, 1):
        rows = view[s["table"][0, j][row, pos // P].long(), pos % P]
        out.append(_values(rows, hkv, d, s["tdt"], j == 1).to(s["tdt"]).view(-1, hkv * d))
    return {"k": out[0], "v": out[1]}


def _plain_store(s):
    c, T, P, ng = s["case"], s["T"], s["P"], s["ng"]
    d, tdt = c["head_dim"], s["tdt"]
    x, y = s["q"].float().view(T, -1, d), s["k"].double().view(T, -1, d)
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["qw"].float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["kw"].double()
    req, pos = _positions(s)
    view, row = _row_view(s), s["rows"].long()[req]
    for j, z in ((0, _rotate(y, s, pos)), (1, s["v"].double().view(T, -1, d))):
        at = s["table"][0, j][row, pos // P].long()
        view[at, pos % P] = _rows(*_quantise(z, c["dtype"], ng), tdt, s["rb"], j == 1)
    return {"q": _rotate(x, s, pos).to(tdt).view(T, -1), **_plain_read(s)}


def _plain_attend(s):
    c, P, T, R = s["case"], s["P"], s["T"], s["R"]
    d, hq, hkv = c["head_dim"], c["heads_q"], c["heads_kv"]
    ctx, new, rows = s["ctx"].long(), s["new"].long(), s["rows"].long()
    longest, most = s["max_blocks"] * P, s["max_new"]
    at = torch.arange(longest, device=DEV)
    pages = s["table"][0][:, rows].clamp(min=0).long()                       # [2, R, blocks]
    view = _row_view(s)
    held = (at < (ctx + new)[:, None])[:, :, None, None]
    k, v = (torch.where(held, _values(view[pages[j][:, at // P], at % P], hkv, d, s["tdt"], j == 1), 0.0) for j in (0, 1))
    i = torch.arange(most, device=DEV)
    start = torch.cumsum(new, 0) - new
    q = s["q"].float()[(start[:, None] + i).clamp(max=T - 1)].view(R, most, hkv, hq // hkv, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(R, hkv, -1, d)                      # rows: head of the group, token
    w = q @ k.permute(0, 2, 3, 1) * s["scale"]
    if c["softcap"]:
        w = c["softcap"] * torch.tanh(w / c["softcap"])
    seen = at <= (ctx[:, None] + i)[:, :, None]                              # [R, most, longest]
    w = w.view(R, hkv, hq // hkv, most, longest).masked_fill(~seen[:, None, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = (w / w.sum(-1, keepdim=True)).view(R, hkv, -1, longest)
    o = (w @ v.permute(0, 2, 1, 3)).view(R, hkv, hq // hkv, most, d).permute(0, 3, 1, 2, 4).reshape(R, most, hq * d)
    req, pos = _positions(s)
    return o[req, pos - ctx[req]].to(s["tdt"])


def run(s):
    c = s["case"]
    if not own:
        return {"store": _plain_store, "read": _plain_read, "attend": _plain_attend}[c["op"]](s)
    kv = s["kv"]
    if c["op"] == "attend":
        kv.attend(s["batch"], 0, s["q"], s["out"], scale=s["scale"], softcap=c["softcap"])
        return s["out"]
    if c["op"] == "store":
        kv.append(s["batch"], 0, s["q"], s["k"], s["v"], q_out=s["q_out"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
    kv.read(0, s["at_row"], s["at_pos"], s["k_read"], s["v_read"])
    got = {"k": s["k_read"], "v": s["v_read"]}
    return {"q": s["q_out"], **got} if c["op"] == "store" else got


# ---- the definitions in 64 bits, request by request ---------------------------------------------


def _exact_rows(s, j, row, p):
    """What the stored rows of positions p of a table row stand for, group by group: [len(p), heads, d]."""
    c, ng = s["case"], s["ng"]
    d, hkv = c["head_dim"], c["heads_kv"]
    page = s["table"][0, j, row].long()[p // s["P"]]
    flat = s["buf"].view(-1).view(torch.uint8)
    base = page * (2 * c["page_elems"]) + (p % s["P"]) * s["rb"]
    out = torch.zeros((p.numel(), hkv, ng, 32), dtype=torch.float64, device=DEV)
    h = torch.arange(hkv, device=DEV)
    for g in range(ng):
        at = base[:, None] + hkv * 16 * ng + (h * ng + g) * 2
        M = (flat[at].int() | flat[at + 1].int() << 8).to(torch.int16).view(s["tdt"]).double()
        for r in range(32):
            if j == 0:                       # words of 8 elements, pairs (2i, 2i + 1) 16 bits apart
                byte, high = ((r // 8) * ng + g) * 4 + (r % 8) // 4 + 2 * (r % 2), (r % 8) // 2 % 2
            else:                            # 16 bits for 4 elements
                byte, high = ((r // 4) * ng + g) * 2 + (r % 4) // 2, r % 2
            code = flat[base[:, None] + h * 16 * ng + byte] >> (4 * high) & 15
            out[:, :, g, r] = (code.double() - 7) * M / 8
    return out.flatten(-2)[..., :d]


def _exact_quantised(x, dtype):
    """x [n, heads, d] after a pass through 4 bits."""
    out = torch.empty_like(x)
    for g in range(0, x.shape[-1], 32):
        y = x[..., g: g + 32]
        top = y.gather(-1, y.abs().argmax(-1, keepdim=True))
        top = torch.where((y == top.abs()).any(-1, keepdim=True), top.abs(), top)
        bits = top.abs().contiguous().view(torch.int64)                      # rounded up to four bits after the first
        M = ((bits + (1 << 48) - 1) >> 48 << 48).view(torch.float64)
        M = (torch.ceil(M / FINEST[dtype]) * FINEST[dtype]).clamp(max=LARGEST[dtype]) * torch.sign(top)
        n = torch.floor((16 * y + M) / (2 * M))
        out[..., g: g + 32] = torch.where(M == 0, 0.0, n.clamp(-7, 8) * M / 8)
    return out


def exact(c, seed):
    s = prepare(c, seed)
    d, hq, hkv = c["head_dim"], c["heads_q"], c["heads_kv"]
    ctx, new = _lengths(c)
    if c["op"] == "read":
        got = {}
        for j, name in ((0, "k"), (1, "v")):
            got[name] = torch.cat([_exact_rows(s, j, int(s["rows"][r]), torch.arange(a + n, device=DEV))
                                   for r, (a, n) in enumerate(zip(ctx, new))]).view(-1, hkv * d)
        return got
    t0 = 0
    if c["op"] == "store":
        outs = {"q": [], "k": [], "v": []}
        for a, n in zip(ctx, new):
            ang = torch.arange(a, a + n, device=DEV).double()[:, None, None] * torch.tensor(
                s["inv_freq"], dtype=torch.float64, device=DEV)
            turn = torch.polar(torch.ones_like(ang), ang)
            for name, w, heads in (("q", s["qw"], hq), ("k", s["kw"], hkv)):
                x = s[name][t0: t0 + n].double().reshape(n, heads, d)
                if w is not None:
                    x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + EPS) * w.double()
                head = x[..., : c["rot"]]
                if c["interleaved"]:
                    z = torch.view_as_complex(head.reshape(n, heads, -1, 2).contiguous()) * turn
                    head = torch.view_as_real(z).reshape(n, heads, -1)
                else:
                    z = torch.complex(head[..., : c["rot"] // 2], head[..., c["rot"] // 2:]) * turn
                    head = torch.cat([z.real, z.imag], -1)
                outs[name].append(torch.cat([head, x[..., c["rot"]:]], -1))
            outs["v"].append(s["v"][t0: t0 + n].double().reshape(n, hkv, d))
            t0 += n
        q, k, v = (torch.cat(outs[name]) for name in "qkv")
        return {"q": q.view(s["T"], -1), "k": _exact_quantised(k, c["dtype"]).view(s["T"], -1),
                "v": _exact_quantised(v, c["dtype"]).view(s["T"], -1)}
    out = torch.empty((s["T"], hkv, hq // hkv, d), dtype=torch.float64, device=DEV)
    for r, (a, n) in enumerate(zip(ctx, new)):
        p = torch.arange(a + n, device=DEV)
        k, v = (_exact_rows(s, j, int(s["rows"][r]), p) for j in (0, 1))
        q = s["q"][t0: t0 + n].double().view(n, hkv, hq // hkv, d)
        x = torch.einsum("nhgd,lhd->hgnl", q, k) / math.sqrt(d)
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        x = torch.where(p <= a + torch.arange(n, device=DEV)[:, None], x, -math.inf)
        out[t0: t0 + n] = torch.einsum("hgnl,lhd->nhgd", torch.softmax(x, -1), v)
        t0 += n
    return out.view(s["T"], hq * d)
