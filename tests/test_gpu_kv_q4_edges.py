"""Edges of key-value caches held in 4 bits on the GPU: missing pages, values that
are not finite, scales and queries of every size, repeatability, graphs, caches
side by side, other streams.  Tolerances as in tests/test_gpu_kv_q4.py.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv as okv
from oracle import kv_q4 as oq4
from tests.test_gpu_kv_q4 import S, TDT, U, Setup, _attend, _check, f64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["K", "V", "KV"])
@pytest.mark.parametrize("dtype,hq,hkv,d,H", [("f16", 4, 2, 64, 320), ("bf16", 5, 1, 128, 120), ("f16", 3, 3, 96, 256),
                                              ("bf16", 2, 2, 256, 300 // 8 * 8), ("f16", 4, 4, 128, 440)])
def test_entries_that_name_no_page(S, which, dtype, hq, hkv, d, H):  # noqa: F811
    """A table entry within a request's length that names no page is reported, its tokens
    get no weight, and no other memory stands in for them (page 0 holds NaN); the other
    requests keep their bits."""
    ctx, new = [700, 300, 600, 5, 2000, 90, 60], [1, 40, 150, 9, 1, 1, 30]
    s = Setup(S, ctx, new, hq, hkv, d, H, dtype, seed=26, first_page=1)
    s.pool.buffer[0].view(torch.int16).fill_(-1)
    s.oracle_plan()
    full = s.fill()
    b, q, out = _attend(s, full)
    good = out.clone()
    blocks_of = lambda lo, hi: list(range(lo // s.P + 1, hi // s.P))  # noqa: E731
    last = [(c + n - 1) // s.P for c, n in zip(ctx, new)]
    holes = {0: [0, last[0] // 2], 1: [1, last[1] - 1], 2: blocks_of(128, 300), 4: [last[4] - 2],
             5: list(range(last[5] + 1)), 6: list(range(last[6] + 1))}      # 5 and 6: nothing is left
    for r, blocks in holes.items():
        for i, blk in enumerate(blocks):
            for j in (0, 1):
                if "KV"[j] in which:
                    s.kv.table[0, j, int(s.rows[r]), blk] = [-1, s.num_pages, -7, 1 << 30][i % 4]
    s.kv.attend(b, 0, q, out[:, : hq * d])
    assert s.pool.status() == S.ERR_INVALID and s.pool.status() == S.OK
    t0 = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        got = out[t0: t0 + n, : hq * d]
        if r not in holes:
            assert torch.equal(got, good[t0: t0 + n, : hq * d]), r
        elif r in (5, 6):
            assert not got.any(), r
        else:
            held = np.array([p for p in range(c + n) if p // s.P not in holes[r]])
            keys, vals = (x[held] for x in full[r])
            qq = f64(q[t0: t0 + n]).reshape(n, hq, d)
            want = np.concatenate([okv.attend(qq[i: i + 1], keys[held <= c + i], vals[held <= c + i],
                                              int((held <= c + i).sum()) - 1, d ** -0.5, 0.0) for i in range(n)])
            err = np.abs(f64(got).reshape(n, hq, d) - want)
            assert (err <= U[dtype] * np.abs(want) + (2.0 ** -12 + U[dtype]) * np.abs(vals).max()).all(), (r, err.max())
        t0 += n
    s.close()


def test_a_missing_page_stores_nothing(S):  # noqa: F811
    s = Setup(S, [0, 4], [6, 3], 2, 2, 64, 150 // 8 * 8, "f16")
    s.opened[:2] = [s.num_pages, -3]
    before = s.pool.buffer.view(torch.int16).clone()
    b = s.plan()
    assert s.pool.status() == S.ERR_INVALID
    x = s.randn(s.T, 128)
    s.kv.append(b, 0, x.clone(), x, x)
    assert s.pool.status() == S.OK
    slots = b.slots.cpu().numpy()
    changed = (s.pool.buffer.view(torch.int16) != before).any(-1).nonzero().flatten().tolist()
    assert (slots == -1).sum() > 0 and sorted(set((slots[slots >= 0] // s.P).tolist())) == changed
    s.close()


@pytest.mark.parametrize("new", [1, 40])
def test_one_request_not_finite_leaves_the_others(S, new):  # noqa: F811
    s = Setup(S, [50, 60, 10], [1, new, 1], 4, 2, 128, 320, "f16", seed=4)
    s.oracle_plan()
    b, q, out = _attend(s, s.fill())
    good, view = out.clone(), s.row_view()
    for j, p in ((0, 9), (1, 5)):                  # M of every group: NaN
        page, at = (int(x[p]) for x in s.at(1, 0, j))
        view[page, at, 2 * 64: 2 * 64 + 16] = 255
    s.kv.attend(b, 0, q, out[:, : s.hq * s.d])
    torch.cuda.synchronize()
    assert torch.equal(out[:1], good[:1]) and torch.equal(out[1 + new:], good[1 + new:])
    assert out[1: 1 + new, : s.hq * s.d].isnan().any()
    s.close()


@pytest.mark.parametrize("dtype,low,high", [("f16", -20, 15), ("f16", -21, -9), ("bf16", -60, 60), ("bf16", -95, -70),
                                            ("bf16", 90, 120)])
@pytest.mark.parametrize("hq,hkv,new", [(4, 4, 1), (8, 1, 1), (4, 1, 1), (4, 2, 60)])
def test_scales_of_every_size(S, dtype, low, high, hq, hkv, new):  # noqa: F811
    """Groups of values from very small to very large ones, growing along the cache, against
    each head's largest value."""
    d = 128
    s = Setup(S, [300, 2000], [new, new], hq, hkv, d, 640, dtype, seed=8)
    s.oracle_plan()
    view, held = s.row_view(), []
    for r in range(2):
        n, got = s.ctx[r] + s.new[r], []
        for j in (0, 1):
            k = s.rng.integers(-7, 9, (n, hkv, d))
            e = np.zeros((n, hkv, 4)) if j == 0 else np.sort(s.rng.uniform(low, high, (n, 1, 1)), 0) + s.rng.uniform(
                -1, 0, (n, hkv, 4))
            M = np.vectorize(lambda m: oq4.scale(m, dtype), otypes=[np.float64])(2.0 ** e * s.rng.choice([-1.0, 1.0], e.shape))
            view[s.at(r, 0, j)] = torch.from_numpy(oq4.pack(k, M, dtype, j == 1)).cuda()
            got.append(oq4.values(k, M, d))
        held.append(got)
    _attend(s, held)
    s.close()


@pytest.mark.parametrize("dtype,size", [("f16", 2.0 ** -20), ("f16", 2.0 ** 14), ("bf16", 2.0 ** -100), ("bf16", 2.0 ** 100)])
@pytest.mark.parametrize("new", [1, 50])
def test_queries_of_every_size(S, dtype, size, new):  # noqa: F811
    """Queries far from one, with a scale that brings their scores back."""
    s = Setup(S, [400, 33], [new, new], 4, 2, 128, 640, dtype, seed=9)
    s.oracle_plan()
    held = s.fill()
    b = s.plan()
    # (held within 3.9: four times 2^14 would be no fp16 number)
    q = (torch.randn(s.T, 512, generator=s.g, device="cuda").double().clamp(-3.9, 3.9) * size).to(TDT[dtype])
    out = torch.full((s.T, 520), 3.0, dtype=TDT[dtype], device="cuda")
    scale = 0.2 / size if dtype == "f16" else float(np.float32(0.2 / size))
    s.kv.attend(b, 0, q, out[:, :512], scale=scale)
    assert s.pool.status() == S.OK
    _check(s, held, q, out, scale=scale)
    # one element far above the rest of its row
    q[:, 7] = size * (2.0 if dtype == "f16" else 2.0 ** 20)
    s.kv.attend(b, 0, q, out[:, :512], scale=scale * (1.0 if dtype == "f16" else 2.0 ** -20))
    _check(s, held, q, out, scale=scale * (1.0 if dtype == "f16" else 2.0 ** -20))
    s.close()


@pytest.mark.parametrize("new", [1, 64])
def test_peaked_and_equal_scores(S, new):  # noqa: F811
    """One key far above the rest gives its value exactly; keys that are all the same."""
    s = Setup(S, [130], [new], 2, 2, 128, 320, "f16", seed=9)
    s.oracle_plan()
    n = 130 + new
    k, M = np.zeros((n, 2, 128), np.int64), np.ones((n, 2, 4))
    k[17, 0], k[:, 1], M[17, 0] = 8, 8, 8.0
    s.row_view()[s.at(0, 0, 0)] = torch.from_numpy(oq4.pack(k, M, "f16", False)).cuda()
    kv_ = s.rng.integers(-7, 9, (n, 2, 128)), np.full((n, 2, 4), 1.5)
    s.row_view()[s.at(0, 0, 1)] = torch.from_numpy(oq4.pack(*kv_, "f16", True)).cuda()
    b = s.plan()
    q = torch.full((new, 256), 8.0, dtype=torch.float16, device="cuda")
    out = torch.full((new, 264), 3.0, dtype=torch.float16, device="cuda")
    s.kv.attend(b, 0, q, out[:, :256])
    torch.cuda.synchronize()
    vals = oq4.values(*kv_, 128)
    assert np.array_equal(f64(out[:, :128]), np.tile(vals[17, 0], (new, 1)))
    _check(s, [(oq4.values(k, M, 128), vals)], q, out)
    s.close()


def test_attend_is_repeatable(S):  # noqa: F811
    s = Setup(S, [3000, 5, 900, 0], [1, 1, 1, 500], 8, 2, 128, 640, "bf16", seed=6)
    s.oracle_plan()
    b, q, out = _attend(s, s.fill())
    first = out.clone()
    for _ in range(5):
        s.kv.attend(b, 0, q, out[:, : s.hq * s.d])
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    s.close()


def test_rows_that_share_a_prefix(S):  # noqa: F811
    """A row that starts with another row's entries attends over, and reads, the shared tokens."""
    s = Setup(S, [42, 42], [1, 9], 4, 2, 64, 320, "f16", spare_rows=1)
    n = 42 // s.P
    s.table[:, :, s.rows[1], :n] = s.table[:, :, s.rows[0], :n]
    s.kv.table.copy_(torch.from_numpy(s.table))
    s.oracle_plan()
    held = s.fill()
    for j in (0, 1):                               # (request 1's fill wrote the shared pages last)
        held[0][j][: n * s.P] = held[1][j][: n * s.P]
    _attend(s, held)
    k = torch.empty(2, 128, dtype=torch.float16, device="cuda")
    s.kv.read(0, s.dev(s.rows), s.dev([3, 3]), k)
    assert torch.equal(k[0], k[1]) and np.array_equal(f64(k[0]).reshape(2, 64), held[0][0][3])
    s.close()


def _plain_codes(x, dtype):
    """x [n, heads, d] in fp64 on the GPU after a pass through 4 bits, vectorised."""
    y = x.unflatten(-1, (-1, 32))
    hi, lo = y.amax(-1, keepdim=True), y.amin(-1, keepdim=True)
    m = torch.where(hi >= -lo, hi, lo)
    e = torch.frexp(m.abs()).exponent.long()
    unit = ((e + (1023 - 5)) << 52).view(torch.float64).clamp(min=oq4.FINEST[dtype])
    M = torch.copysign(torch.ceil(m.abs() / unit) * unit, m)
    k = torch.floor(8 * y / M + 0.5).clamp(-7, 8)
    return (k * M / 8).flatten(-2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("norm,inter,rot", [(False, False, 128), (False, True, 64), (True, False, 128), (True, True, 128)])
def test_codes_of_many_keys(S, dtype, norm, inter, rot):  # noqa: F811
    """Four million normed or rotated elements, among them hundreds so close to a border
    between two codes, or between two M, that fp32 does not tell: every code is that of
    the formula in fp64.  (But for a tie between two signs that the norm's rounding in fp64
    decides: elements whose products with their weights are equal.)"""
    T, hkv, d = 4096, 8, 128
    pool = S.Pool(2 * T // 17 + 40, 5120, dtype, [(8, 8)], 1, 1, T, device=torch.device("cuda", 0))
    kv = S.KVCache(pool, 1, hkv, hkv, d, 1, T // 17 + 9, bits=4)
    freq = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    kv.set_rotary(rot, freq, interleaved=inter, mscale=1.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx = 100 // 17 * 17
    kv.table[0, :, 0, : ctx // 17] = 0
    n_blocks = -(-(ctx + T) // 17) - ctx // 17
    b = kv.plan(torch.tensor([ctx], **i32), torch.tensor([T], **i32), torch.arange(1, 2 * n_blocks + 1, **i32), T, T)
    g = torch.Generator(device="cuda").manual_seed(11)
    k = torch.randn(T, hkv * d, generator=g, device="cuda").to(TDT[dtype])
    w = (torch.randn(d, generator=g, device="cuda") * 0.2 + 1).to(TDT[dtype]) if norm else None
    kv.append(b, 0, k.clone(), k, k, q_out=torch.empty_like(k), q_weight=w, k_weight=w, eps=2.0 ** -20)
    got, vals = torch.empty_like(k), torch.empty_like(k)
    pos = torch.arange(ctx, ctx + T, **i32)
    kv.read(0, torch.zeros_like(pos), pos, got, vals)
    assert pool.status() == S.OK
    assert torch.equal(vals.double().view(T, hkv, d), _plain_codes(k.double().view(T, hkv, d), dtype))
    x = k.double().view(T, hkv, d)
    if norm:
        rs = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 2.0 ** -20)
        x = x * w.double() * rs
    ang = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    c, s_ = torch.cos(ang), torch.sin(ang)
    a, bb = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    u, v = a * c - bb * s_, a * s_ + bb * c
    y = torch.cat([torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1), x[..., rot:]], -1)
    assert torch.equal(got.double().view(T, hkv, d), _plain_codes(y, dtype))
    kv.close()
    pool.close()


def test_step_in_a_cuda_graph(S):  # noqa: F811
    """plan, append, attend and read captured once and replayed for steps of other lengths,
    rows and pages: the same bits as the calls made one by one."""
    hq, hkv, d, T = 8, 2, 64, 40
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        pool = S.Pool(400, 320, "f16", [(8, 8)], 1, 1, T, device=torch.device("cuda", 0), compute_stream=stream)
        kv = S.KVCache(pool, 1, hq, hkv, d, 6, 40, bits=4)
        P = kv.tokens_per_page
        kv.set_rotary(d, [1.0 / (i + 1) for i in range(d // 2)])
        pool.buffer.zero_()
        i32 = dict(dtype=torch.int32, device="cuda")
        ctx, new, rows = torch.zeros(3, **i32), torch.zeros(3, **i32), torch.arange(3, **i32)
        pages = torch.zeros(60, **i32)
        qkv = torch.zeros(T, (hq + 2 * hkv) * d, dtype=torch.float16, device="cuda")
        q_out, out = (torch.zeros(T, hq * d, dtype=torch.float16, device="cuda") for _ in range(2))
        at_row, at_pos = torch.zeros(T, **i32), torch.full((T,), -1, **i32)
        k_out, v_out = (torch.zeros(T, hkv * d, dtype=torch.float16, device="cuda") for _ in range(2))
        w = [hq * d, hkv * d, hkv * d]

        def step():
            b = kv.plan(ctx, new, pages, T, 30, rows=rows)
            q, k, v = qkv.split(w, 1)
            kv.append(b, 0, q, k, v, q_out=q_out)
            kv.attend(b, 0, q_out, out)
            kv.read(0, at_row, at_pos, k_out, v_out)

        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        g = torch.Generator(device="cuda").manual_seed(3)
        used = 1
        held = {r: 0 for r in range(6)}
        for rr, nn in (([0, 1, 2], [30, 5, 1]), ([2, 0, 5], [1, 1, 20]), ([5, 2, 1], [1, 12, 3])):
            c = [held[r] for r in rr]
            opened = sum(-(-(a + n) // P) - -(-a // P) for a, n in zip(c, nn))
            ctx.copy_(torch.tensor(c, dtype=torch.int32)); new.copy_(torch.tensor(nn, dtype=torch.int32))
            rows.copy_(torch.tensor(rr, dtype=torch.int32))
            pages[: 2 * opened] = torch.arange(used, used + 2 * opened, **i32)
            used += 2 * opened
            qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
            for r, n in zip(rr, nn):
                held[r] += n
            at_row.fill_(rr[1]); at_pos.copy_(torch.arange(T, **i32)); at_pos[held[rr[1]]:] = -1
            table = kv.table.clone()
            graph.replay()
            stream.synchronize()
            got = [x.clone() for x in (out, k_out, v_out, q_out, pool.buffer)]
            kv.table.copy_(table)
            step()
            stream.synchronize()
            assert all(torch.equal(a.view(torch.int16), b.view(torch.int16))
                       for a, b in zip(got, (out, k_out, v_out, q_out, pool.buffer)))
            assert pool.status() == S.OK
        kv.close()
        pool.close()


def test_a_16_bit_and_a_4_bit_cache_in_one_pool(S):  # noqa: F811
    """Both kinds over one pool's pages, planned in turn; a batch serves its own cache only."""
    hq, hkv, d, H = 4, 2, 64, 512
    pool = S.Pool(60, H, "f16", [(8, 8)], 1, 1, 64, device=torch.device("cuda", 0))
    pool.buffer.view(torch.int16).fill_(-1)
    c16, c4 = S.KVCache(pool, 1, hq, hkv, d, 2, 10), S.KVCache(pool, 1, hq, hkv, d, 2, 10, bits=4)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(20, n * d, generator=g, device="cuda").half() for n in (hq, hkv, hkv))
    b16 = c16.plan(i32([0]), i32([20]), i32(range(10)), 20, 20)
    c16.append(b16, 0, q.clone(), k, v)
    b4 = c4.plan(i32([0]), i32([20]), i32(range(20, 30)), 20, 20)
    c4.append(b4, 0, q.clone(), k, v)
    out16, out4 = torch.empty_like(q), torch.empty_like(q)
    c16.attend(b16, 0, q, out16)
    c4.attend(b4, 0, q, out4)
    for call in (lambda: c16.attend(b4, 0, q, out16), lambda: c4.attend(b16, 0, q, out4),
                 lambda: c4.append(b16, 0, q, k, v, q_out=out4)):
        with pytest.raises(S.SloraError) as e:
            call()
        assert e.value.code == S.ERR_INVALID
    for cache, out, tol in ((c16, out16, 0.0), (c4, out4, 1.0)):
        kk, vv = torch.empty_like(k), torch.empty_like(v)
        cache.read(0, i32([0] * 20), i32(range(20)), kk, vv)
        want = okv.attend(f64(q).reshape(20, hq, d), f64(kk).reshape(20, hkv, d), f64(vv).reshape(20, hkv, d), 0, d ** -0.5, 0.0)
        err = np.abs(f64(out).reshape(20, hq, d) - want)
        assert (err <= U["f16"] * np.abs(want) + (2.0 ** -12 + U["f16"]) * np.abs(f64(vv)).max()).all()
        if not tol:
            assert torch.equal(kk, k) and torch.equal(vv, v)
    assert pool.status() == S.OK
    c16.close()
    c4.close()
    pool.close()


def test_refusals(S):  # noqa: F811
    s = Setup(S, [5], [2], 4, 2, 64, 320, "f16")
    b = s.plan()
    x, q = s.randn(2, 128), s.randn(2, 256)
    rows, pos = s.dev([int(s.rows[0])] * 2), s.dev([0, 1])
    k, v = torch.empty_like(x), torch.empty_like(x)
    h = s.kv.handle

    def refused(call, error=S.SloraError):
        with pytest.raises(error):
            call()
        assert s.pool.status() == S.OK

    refused(lambda: s.kv.read(1, rows, pos, k, v))                     # no such layer
    refused(lambda: s.kv.read(0, rows, pos))                           # neither is wanted
    refused(lambda: s.kv.read(0, rows, pos, k, k))                     # one over the other
    refused(lambda: S.slora_kv_read(h, 0, -1, rows.data_ptr(), pos.data_ptr(), k.data_ptr(), 128, 0, 0))
    refused(lambda: S.slora_kv_read(h, 0, 2, 0, pos.data_ptr(), k.data_ptr(), 128, 0, 0))
    refused(lambda: S.slora_kv_read(h, 0, 2, rows.data_ptr() + 2, pos.data_ptr(), k.data_ptr(), 128, 0, 0))
    refused(lambda: S.slora_kv_read(h, 0, 2, rows.data_ptr(), pos.data_ptr(), k.data_ptr() + 8, 128, 0, 0))
    refused(lambda: S.slora_kv_read(h, 0, 2, rows.data_ptr(), pos.data_ptr(), k.data_ptr(), 120, 0, 0))
    refused(lambda: S.slora_kv_read(h, 0, 2, rows.data_ptr(), pos.data_ptr(), k.data_ptr(), 132, 0, 0))
    refused(lambda: s.kv.read(0, rows, pos[:1], k, v), ValueError)
    refused(lambda: s.kv.read(0, rows.long(), pos, k, v), ValueError)
    refused(lambda: s.kv.read(0, rows, pos, k[:1], v), ValueError)
    refused(lambda: s.kv.read(0, rows, pos, k.float(), v), ValueError)
    refused(lambda: s.kv.append(b, 0, q, x, x, q_out=q[:, :], q_weight=x[0, :64]))
    refused(lambda: s.kv.attend(b, 0, q, q))
    s.close()
    pool = S.Pool(8, 72, "f16", [(8, 8)], 1, 1, 4, device=torch.device("cuda", 0))     # 144 bytes a page
    for bad in (dict(heads_kv=2, head_dim=128), dict(heads_kv=1, head_dim=264), dict(heads_kv=1, head_dim=24),
                dict(heads_kv=5, head_dim=64), dict(heads_kv=1, head_dim=128, max_blocks=0)):
        args = dict(layers=1, heads_q=bad["heads_kv"], max_requests=2, max_blocks=4) | bad
        if bad == dict(heads_kv=2, head_dim=128):
            S.KVCache(pool, **args, bits=4).close()                                    # just fits
            args["heads_q"] = args["heads_kv"] = 4
        with pytest.raises(S.SloraError) as e:
            S.KVCache(pool, **args, bits=4)
        assert e.value.code == S.ERR_INVALID
    pool.close()


def test_timing_names_the_read_kernel(S):  # noqa: F811
    s = Setup(S, [30], [1], 4, 4, 64, 320, "f16")
    s.oracle_plan()
    s.fill()
    S.slora_timing_enable(s.pool.handle, True)
    k = torch.empty(3, 256, dtype=torch.float16, device="cuda")
    s.kv.read(0, s.dev([int(s.rows[0])] * 3), s.dev([0, 1, 2]), k)
    t = S.slora_timing_read(s.pool.handle)
    assert t["kv_read"][1] == 1 and t["kv_read"][0] > 0 and t["kv_append"][1] == 0
    s.close()


@pytest.mark.slow
def test_debug_build_catches_planted_indices():
    """The SLORA_DEBUG build, in a process of its own."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "tests", "debug_kv_q4_check.py")], capture_output=True, text=True,
                       env={**os.environ, "SLORA_DEBUG": "1"}, cwd=root, timeout=600)
    assert r.returncode == 0 and "debug build OK" in r.stdout, r.stdout + r.stderr
