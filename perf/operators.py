"""Measured cases of the paged key-value cache operators: plan, append, attend.

``plan``    block-table entries and slot map of a step's tokens, from the
            requests' lengths.
``append``  per-head RMS norm of queries and keys (optional), rotary positions,
            and the store of keys and values into their slots of the page pool.
``attend``  causal attention of every request's new tokens (one in decode, a
            chunk in prefill) over its paged keys and values.

A page holds whole tokens: P = page_elems / (heads_kv * head_dim) of them, so
that the pool's buffer is also a matrix of token rows, and position t of a
request sits in row page(t // P) * P + t % P.  Keys and values have pages of
their own, in every layer.

The plain forms are elementary torch operations in 32 bits, rounded once at
the end; ``exact`` restates the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def _mha7b(**kw):
    """The 7B-shaped layer: 32 heads of 128, a page (4096) is one token's K or V."""
    return dict(heads_q=32, heads_kv=32, head_dim=128, page_elems=4096, dtype="f16", **kw)


def _gqa13b(**kw):
    """A 13B-shaped layer (hidden size 5120, 40 heads) with 8 shared key heads: five tokens a page."""
    return dict(heads_q=40, heads_kv=8, head_dim=128, page_elems=5120, dtype="bf16", **kw)


def listed():
    return [
        # the serving trace's full decode batch: one token each, 32 layers' tables
        dict(name="plan_decode", op="plan", layers=32, decode=256, ctx_lo=8, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, **_mha7b()),
        # a prefill batch of 32 prompts of 8..512 tokens, every block new
        dict(name="plan_prefill", op="plan", layers=32, decode=0, ctx_lo=0, ctx_hi=0, chunks=32, new_lo=8, new_hi=512,
             chunk_ctx=0, **_mha7b()),
        # a single request's decode step, where latency counts
        dict(name="append_one", op="append", layers=1, decode=1, ctx_lo=640, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, norm=False, interleaved=False, rot=128, factor=1.0, **_mha7b()),
        # the trace's decode batch, whole-head rotary of the half layout
        dict(name="append_decode", op="append", layers=1, decode=256, ctx_lo=8, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, norm=False, interleaved=False, rot=128, factor=1.0, **_mha7b()),
        # the prefill batch with normed heads, an interleaved rotary of half the
        # head, and positions stretched by four for a long context
        dict(name="append_prefill_norm", op="append", layers=1, decode=0, ctx_lo=0, ctx_hi=0, chunks=32, new_lo=8,
             new_hi=512, chunk_ctx=8191, norm=True, interleaved=True, rot=64, factor=4.0, **_gqa13b()),
        # one request, one token: the smallest attention call
        dict(name="decode_one", op="attend", layers=1, decode=1, ctx_lo=640, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, softcap=0.0, **_mha7b()),
        # the trace's decode batch
        dict(name="decode_batch", op="attend", layers=1, decode=256, ctx_lo=8, ctx_hi=640, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, softcap=0.0, **_mha7b()),
        # shared key heads, contexts of very different lengths, pages of five tokens
        dict(name="decode_gqa", op="attend", layers=1, decode=128, ctx_lo=17, ctx_hi=8192, chunks=0, new_lo=0, new_hi=0,
             chunk_ctx=0, softcap=0.0, **_gqa13b()),
        # one request with a very long context, scores capped: all of the GPU on one row
        dict(name="decode_long_capped", op="attend", layers=1, decode=1, ctx_lo=131071, ctx_hi=131071, chunks=0,
             new_lo=0, new_hi=0, chunk_ctx=0, softcap=30.0, **_gqa13b()),
        # the prefill batch: 32 whole prompts
        dict(name="chunk_prefill", op="attend", layers=1, decode=0, ctx_lo=0, ctx_hi=0, chunks=32, new_lo=8, new_hi=512,
             chunk_ctx=0, softcap=0.0, **_mha7b()),
        # a chunk of a long prompt over what earlier chunks stored
        dict(name="chunk_long", op="attend", layers=1, decode=0, ctx_lo=0, ctx_hi=0, chunks=1, new_lo=1024, new_hi=1024,
             chunk_ctx=16383, softcap=0.0, **_gqa13b()),
        # the trace's mixed step: decode tokens and prompt chunks within 1024 tokens
        dict(name="step_mixed", op="attend", layers=1, decode=200, ctx_lo=8, ctx_hi=640, chunks=4, new_lo=100,
             new_hi=312, chunk_ctx=0, softcap=0.0, **_mha7b()),
    ]


def _log(rng, lo, hi):
    """An odd whole number, spread over the logarithm of lo..hi."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))) | 1


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "attend"])
    heads_kv, group = rng.choice([1, 2, 4, 5, 8, 8]), rng.choice([1, 2, 4, 5, 7, 8])
    if rng.random() < 0.3:
        heads_kv, group = rng.choice([20, 32, 40]), 1
    d = rng.choice([64, 80, 128, 128])
    per_page = rng.choice([1, 2, 4, 5, 16])
    while heads_kv * d * per_page > 8192:
        per_page = max(1, per_page // 2)
    c = dict(op=op, layers=_log(rng, 1, 32) if op == "plan" else 1, heads_q=heads_kv * group, heads_kv=heads_kv,
             head_dim=d, page_elems=heads_kv * d * per_page, dtype=rng.choice(["f16", "bf16"]))
    kind = rng.choice(["decode", "decode", "chunk", "mixed"])
    # at most about 200 M cached elements a side (decode) and 10^10 scores times heads (chunks)
    hi = _log(rng, 17, 32767)
    most = max(1, 200_000_000 // (heads_kv * d * hi))
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
    if op == "plan":
        c["ctx_hi"] = min(c["ctx_hi"], 2047)
        c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
    if op == "append":
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


def work(c):
    ctx, new = _lengths(c)
    T, R, L2 = sum(new), len(new), 2 * c["layers"]
    d, hq, hkv = c["head_dim"], c["heads_q"], c["heads_kv"]
    P = c["page_elems"] // (hkv * d)
    if c["op"] == "plan":
        fresh = sum(-(-(a + n) // P) + (-a // P) for a, n in zip(ctx, new))
        old = T - fresh if P > 1 else 0          # about: tokens whose block was there already
        return {"bytes": 4 * (3 * R + 2 * R + 1 + 2 * fresh * L2 + max(0, old) * L2 + T * L2 + 2 * T), "flops": 0}
    if c["op"] == "append":
        return {"bytes": T * (4 * d * (hq + 2 * hkv) + 12), "flops": 10 * T * d * (hq + hkv)}
    lens = [a + n for a, n in zip(ctx, new)]
    scores = sum(n * a + n * (n + 1) // 2 for a, n in zip(ctx, new))
    return {"bytes": 4 * T * hq * d + sum(lens) * hkv * d * 4 + sum(8 * -(-n // P) for n in lens),
            "flops": 4 * d * hq * scores}


# ---- inputs -------------------------------------------------------------------------------------


def _inv_freq(c):
    """Rotary frequencies (radians a position) in 64 bits, positions stretched by `factor`."""
    return [10000.0 ** (-2.0 * i / c["rot"]) / c["factor"] for i in range(c["rot"] // 2)]


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    tdt = torch.float16 if c["dtype"] == "f16" else torch.bfloat16
    L, hq, hkv, d, H = c["layers"], c["heads_q"], c["heads_kv"], c["head_dim"], c["page_elems"]
    P = H // (hkv * d)
    ctx, new = _lengths(c)
    R, T = len(new), sum(new)
    i32 = dict(dtype=torch.int32, device=DEV)
    first = torch.tensor([-(-a // P) for a in ctx], device=DEV)            # blocks stored before the step
    total = torch.tensor([-(-(a + n) // P) for a, n in zip(ctx, new)], device=DEV)
    max_blocks = max(1, int(total.max()))
    max_rows = R + 3
    req = torch.repeat_interleave(torch.arange(R, device=DEV), total)
    blk = torch.arange(req.numel(), device=DEV) - (torch.cumsum(total, 0) - total)[req]
    fresh = blk >= first[req]
    # attend reads every block, append writes the new tokens' blocks, plan none: the pool
    # holds the blocks whose contents count, the table names any page for the others
    held = torch.ones_like(fresh) if c["op"] == "attend" else (blk >= torch.tensor([a // P for a in ctx], device=DEV)[req])
    n_held = int(held.sum())
    num_pages = n_held * 2 * L + 5
    s = dict(case=c, P=P, R=R, T=T, num_pages=num_pages, max_rows=max_rows, max_blocks=max_blocks, max_new=max(new))
    s["rows"] = torch.randperm(max_rows, generator=g, device=DEV)[:R].to(torch.int32)   # table row of each request
    s["ctx"], s["new"] = torch.tensor(ctx, **i32), torch.tensor(new, **i32)
    # pages in no order, block by block: [block][layer][K, V]
    pages = torch.randint(num_pages, (req.numel(), L, 2), generator=g, **i32)
    pages[held] = torch.randperm(num_pages, generator=g, device=DEV)[: n_held * 2 * L].to(torch.int32).view(-1, L, 2)
    s["pages"] = pages[fresh].reshape(-1).contiguous()                     # what the step's allocation handed out
    table = torch.full((L, 2, max_rows, max_blocks), -1, **i32)
    known = ~fresh if c["op"] == "plan" else torch.ones_like(fresh)
    table[:, :, s["rows"].long()[req[known]], blk[known]] = pages[known].permute(1, 2, 0)
    s["table"] = table
    if c["op"] == "plan":
        buf = torch.empty((num_pages, H), dtype=tdt, device=DEV) if own else None
    else:
        buf = torch.empty((num_pages, H), dtype=tdt, device=DEV).normal_(generator=g)
    if c["op"] == "append":
        qkv = torch.empty((T, (hq + 2 * hkv) * d), dtype=tdt, device=DEV).normal_(generator=g)   # one fused product's rows
        s["q"], s["k"], s["v"] = qkv[:, : hq * d], qkv[:, hq * d: (hq + hkv) * d], qkv[:, (hq + hkv) * d:]
        s["q_out"] = torch.empty((T, hq * d), dtype=tdt, device=DEV)
        s["qw"] = s["kw"] = None
        if c["norm"]:
            w = torch.empty((2, d), device=DEV).normal_(generator=g) * 0.2 + 1.0
            s["qw"], s["kw"] = w.to(tdt).unbind(0)
        s["inv_freq"] = _inv_freq(c)
        s["inv_freq32"] = torch.tensor(s["inv_freq"], dtype=torch.float32, device=DEV)
    if c["op"] == "attend":
        s["q"] = (torch.empty((T, hq * d), dtype=tdt, device=DEV).normal_(generator=g) * 2.0)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(d)
    s["buf"] = buf
    if own:
        from lora_adapters_gb300 import slora

        pool = slora.Pool(num_pages, H, c["dtype"], [(8, 8)], 1, 1, T, device=torch.device(DEV, torch.cuda.current_device()),
                          buffer=buf)
        kv = slora.KVCache(pool, L, hq, hkv, d, max_rows, max_blocks)
        kv.table.copy_(table)
        s["pool"], s["kv"] = pool, kv
        if c["op"] == "append":
            kv.set_rotary(c["rot"], s["inv_freq"], interleaved=c["interleaved"])
        if c["op"] != "plan":
            s["batch"] = kv.plan(s["ctx"], s["new"], s["pages"], T, s["max_new"], rows=s["rows"])
    if c["op"] == "append":
        s["pos"], s["slots"] = _positions(s)[1], _plain_plan(s)["slots"]
    return s


# ---- plain forms --------------------------------------------------------------------------------


def _positions(s):
    """(request, position) of every new token."""
    new, ctx = s["new"].long(), s["ctx"].long()
    ends = torch.cumsum(new, 0)
    tok = torch.arange(s["T"], device=DEV)
    req = torch.searchsorted(ends, tok, right=True)
    return req, ctx[req] + tok - (ends - new)[req]


def _plain_plan(s):
    c, P = s["case"], s["P"]
    new, ctx, rows, table = s["new"].long(), s["ctx"].long(), s["rows"].long(), s["table"]
    first = (ctx + P - 1) // P
    nb = (ctx + new + P - 1) // P - first
    ends = torch.cumsum(nb, 0)
    pages = s["pages"].view(-1, c["layers"], 2)
    j = torch.arange(pages.shape[0], device=DEV)
    breq = torch.searchsorted(ends, j, right=True)
    table[:, :, rows[breq], first[breq] + j - (ends - nb)[breq]] = pages.permute(1, 2, 0)
    req, pos = _positions(s)
    slots = table[:, :, rows[req], pos // P] * P + (pos % P).to(torch.int32)
    start = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    i32 = torch.int32
    return {"table": table, "slots": slots.to(i32), "tok_req": req.to(i32), "tok_pos": pos.to(i32),
            "q_start": start.to(i32), "kv_len": (ctx + new).to(i32)}


def _rotate(x, s):
    """The rotary turn of x [T, heads, d] in 32 bits."""
    c = s["case"]
    rot = c["rot"]
    ang = s["pos"].float()[:, None] * s["inv_freq32"]
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., : rot // 2], x[..., rot // 2: rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], -1).flatten(-2) if c["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    c, T = s["case"], s["T"]
    d, hkv = c["head_dim"], c["heads_kv"]
    x, y = s["q"].float().view(T, -1, d), s["k"].float().view(T, -1, d)
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["qw"].float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["kw"].float()
    dt = s["q"].dtype
    cache = s["buf"].view(-1, hkv * d)
    slots = s["slots"][0].long()
    cache[slots[0]] = _rotate(y, s).to(dt).view(T, -1)
    cache[slots[1]] = s["v"]
    return {"q": _rotate(x, s).to(dt).view(T, -1), "cache": s["buf"]}


def _plain_attend(s):
    c, P, T, R = s["case"], s["P"], s["T"], s["R"]
    d, hq, hkv = c["head_dim"], c["heads_q"], c["heads_kv"]
    ctx, new, rows = s["ctx"].long(), s["new"].long(), s["rows"].long()
    longest, most = s["max_blocks"] * P, s["max_new"]
    at = torch.arange(longest, device=DEV)
    pages = s["table"][0][:, rows].clamp(min=0).long()                       # [2, R, blocks]
    slots = pages[:, :, at // P] * P + at % P                                # [2, R, longest]
    cache = s["buf"].view(-1, hkv, d)
    held = (at < (ctx + new)[:, None])[:, :, None, None]
    k = torch.where(held, cache[slots[0]].float(), 0.0)
    v = torch.where(held, cache[slots[1]].float(), 0.0)
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
    return o[req, pos - ctx[req]].to(s["q"].dtype)


def run(s):
    c = s["case"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[c["op"]](s)
    kv = s["kv"]
    if c["op"] == "plan":
        b = kv.plan(s["ctx"], s["new"], s["pages"], s["T"], s["max_new"], rows=s["rows"])
        return {"table": kv.table, "slots": b.slots, "tok_req": b.tok_req, "tok_pos": b.tok_pos, "q_start": b.q_start,
                "kv_len": b.kv_len}
    if c["op"] == "append":
        kv.append(s["batch"], 0, s["q"], s["k"], s["v"], q_out=s["q_out"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
        return {"q": s["q_out"], "cache": s["buf"]}
    kv.attend(s["batch"], 0, s["q"], s["out"], scale=s["scale"], softcap=c["softcap"])
    return s["out"]


# ---- the definitions in 64 bits, request by request ---------------------------------------------


def exact(c, seed):
    if c["op"] == "plan":
        return None          # whole numbers only
    s = prepare(c, seed)
    d, hq, hkv, P = c["head_dim"], c["heads_q"], c["heads_kv"], s["P"]
    ctx, new = _lengths(c)
    if c["op"] == "append":
        cache = s["buf"].double().view(-1, hkv, d)
        q_out = torch.empty((s["T"], hq, d), dtype=torch.float64, device=DEV)
        t0 = 0
        for r, (a, n) in enumerate(zip(ctx, new)):
            row = int(s["rows"][r])
            p = torch.arange(a, a + n, device=DEV)
            ang = p.double()[:, None, None] * torch.tensor(s["inv_freq"], dtype=torch.float64, device=DEV)
            turn = torch.polar(torch.ones_like(ang), ang)
            slot = [s["table"][0, j, row].long()[p // P] * P + p % P for j in (0, 1)]
            for x, w, heads, put in ((s["q"], s["qw"], hq, None), (s["k"], s["kw"], hkv, slot[0])):
                x = x[t0: t0 + n].double().reshape(n, heads, d)
                if w is not None:
                    x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + EPS) * w.double()
                head = x[..., : c["rot"]]
                if c["interleaved"]:
                    z = torch.view_as_complex(head.reshape(n, heads, -1, 2).contiguous()) * turn
                    head = torch.view_as_real(z).reshape(n, heads, -1)
                else:
                    z = torch.complex(head[..., : c["rot"] // 2], head[..., c["rot"] // 2:]) * turn
                    head = torch.cat([z.real, z.imag], -1)
                x = torch.cat([head, x[..., c["rot"]:]], -1)
                if put is None:
                    q_out[t0: t0 + n] = x
                else:
                    cache[put] = x
            cache[slot[1]] = s["v"][t0: t0 + n].double().reshape(n, hkv, d)
            t0 += n
        return {"q": q_out.view(s["T"], -1), "cache": cache.view(s["num_pages"], -1)}
    out = torch.empty((s["T"], hkv, hq // hkv, d), dtype=torch.float64, device=DEV)
    cache = s["buf"].view(-1, hkv, d)
    t0 = 0
    for r, (a, n) in enumerate(zip(ctx, new)):
        p = torch.arange(a + n, device=DEV)
        k, v = (cache[s["table"][0, j, int(s["rows"][r])].long()[p // P] * P + p % P].double() for j in (0, 1))
        q = s["q"][t0: t0 + n].double().view(n, hkv, hq // hkv, d)
        x = torch.einsum("nhgd,lhd->hgnl", q, k) / math.sqrt(d)
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        x = torch.where(p <= a + torch.arange(n, device=DEV)[:, None], x, -math.inf)
        out[t0: t0 + n] = torch.einsum("hgnl,lhd->nhgd", torch.softmax(x, -1), v)
        t0 += n
    return out.view(s["T"], hq * d)
