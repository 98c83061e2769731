"""The paged key-value cache operators at their edges, on the GPU against the
fp64 oracle; tolerances are those of tests/test_gpu_kv.py where none is derived
beside the test."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.test_gpu_kv import S, Setup, TDT, U, _check_attend, _fill_and_attend, f64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [50.0, 65.0, 1e3, 1e4, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("dtype,new,d", [("f16", 1, 128), ("bf16", 1, 64), ("f16", 60, 128), ("bf16", 60, 80)])
def test_softcap_far_above_the_scores(S, softcap, dtype, new, d):
    """c(s) keeps the bits of a small s whatever the softcap, in both kernels."""
    s = Setup(S, [300], [new], 4, 4, d, 1, dtype, seed=21)
    _, q, out = _fill_and_attend(S, s, softcap=softcap)
    _check_attend(s, q, out, softcap=softcap)
    s.close()


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("softcap", [2.0, 1e-3, 1e-30, 1e-42])
def test_softcap_below_the_scores(S, new, softcap):
    s = Setup(S, [300], [new], 4, 4, 64, 1, "f16", seed=22)
    _, q, out = _fill_and_attend(S, s, softcap=softcap)
    _check_attend(s, q, out, softcap=softcap)
    s.close()


@pytest.mark.parametrize("new", [1, 60])
def test_softcap_around_large_scores(S, new):
    """Scores from far below softcap to near it (q . k scale of about +-150)."""
    s = Setup(S, [300], [new], 4, 4, 64, 1, "f16", seed=22)
    _, q, out = _fill_and_attend(S, s, softcap=100.0, scale=64 ** -0.5 * 16)
    _check_attend(s, q, out, softcap=100.0, scale=64 ** -0.5 * 16)
    s.close()


@pytest.mark.parametrize("which", ["K", "V", "KV"])
@pytest.mark.parametrize("dtype,hq,hkv,d,P", [("f16", 4, 2, 64, 4), ("bf16", 5, 1, 128, 3), ("f16", 3, 3, 80, 1),
                                               ("bf16", 2, 2, 256, 2)])
def test_entries_that_name_no_page(S, which, dtype, hq, hkv, d, P):
    """A table entry within a request's length that names no page is reported,
    its tokens get no weight, and no other memory stands in for them (page 0
    holds NaN); the other requests keep their bits."""
    ctx, new = [700, 300, 600, 5, 2000, 90, 60], [1, 40, 150, 9, 1, 1, 30]
    s = Setup(S, ctx, new, hq, hkv, d, P, dtype, seed=26, first_page=1)
    s.pool.buffer[0].fill_(float("nan"))
    b, q, out = _fill_and_attend(S, s)
    good = out.clone()
    holes = {0: [0, 5], 1: [2, 30], 2: list(range(128 // P + 1, 256 // P + 1)), 4: [399 // P],
             5: list(range(-(-91 // P))), 6: list(range(-(-90 // P)))}       # 5 and 6: nothing is left
    for r, blocks in holes.items():
        for i, blk in enumerate(blocks):
            for j in (0, 1):
                if "KV"[j] in which:
                    s.kv.table[0, j, int(s.rows[r]), blk] = [-1, s.num_pages, -7, 1 << 30][i % 4]
    s.kv.attend(b, 0, q, out[:, : hq * d])
    assert s.pool.status() == S.ERR_INVALID and s.pool.status() == S.OK
    cache, t0 = s.cache_rows(), 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        if r not in holes:
            assert torch.equal(out[t0: t0 + n], good[t0: t0 + n]), r
        elif r in (5, 6):
            assert not out[t0: t0 + n, : hq * d].any(), r
        else:
            held = np.array([p for p in range(c + n) if p // P not in holes[r]])
            at = torch.from_numpy(held).cuda()
            keys, vals = (f64(cache[s.slot_rows(r, 0, j)[at]]).reshape(-1, hkv, d) for j in (0, 1))
            want = okv.attend(f64(q[t0: t0 + n]).reshape(n, hq, d), keys, vals, held.size - n, d ** -0.5, 0.0)
            got = f64(out[t0: t0 + n, : hq * d]).reshape(n, hq, d)
            vmax = np.repeat(np.abs(vals).max((0, 2)), hq // hkv)[None, :, None]
            err = np.abs(got - want)
            assert (err <= U[dtype] * np.abs(want) + (2.0 ** -12 + U[dtype]) * vmax).all(), (r, err.max())
        t0 += n
    s.close()


@pytest.mark.parametrize("ctx,new", [(40, 1), (3000, 1), (20000, 1), (100, 40), (20000, 16)])
def test_a_query_that_is_not_a_number(S, ctx, new):
    """It makes its own row NaN, wherever its segment is split, and no other."""
    s = Setup(S, [ctx, 7], [new, 1], 4, 2, 64, 4, "f16", seed=24)
    b, q, out = _fill_and_attend(S, s)
    want = out.clone()
    t = new // 2
    want[t, 3 * 64: 4 * 64] = float("nan")
    q[t, 3 * 64 + 5] = float("nan")          # head 3 of one token
    s.kv.attend(b, 0, q, out[:, : 4 * 64])
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(9.0), want.nan_to_num(9.0))
    s.close()


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("heads,ctx,new,first,count", [(2, 1000, 1, 16, 16), (2, 1000, 1, 990, 4), (1, 1000, 1, 0, 1000),
                                                       (2, 40000, 1, 16, 32), (1, 16000, 16, 256, 128),
                                                       (2, 16000, 16, 300, 1), (2, 40, 30, 3, 2)])
def test_keys_that_are_not_numbers(S, heads, ctx, new, first, count, softcap):
    """They reach every row that sees them, also where a part of a split segment
    holds nothing else."""
    s = Setup(S, [ctx, 7], [new, 1], heads, heads, 64, 4, "f16", seed=25)
    b, q, out = _fill_and_attend(S, s, softcap=softcap)
    want = out.clone()
    at = 64 * (heads - 1)                    # the last head's
    want[:new, at: at + 64] = float("nan")
    s.cache_rows()[s.slot_rows(0, 0, 0)[first: first + count], at:] = float("nan")
    s.kv.attend(b, 0, q, out[:, : 64 * heads], softcap=softcap)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(9.0), want.nan_to_num(9.0))
    s.close()


def _long_segments(S, ctx, new, hkv, d, R, dtype, above, sink, rest):
    """R requests over the same ctx + new keys, key 1000 `above` nats over the others, all of
    whose weights are e^-above; its value `sink`, the others' from rest(n, cols).  With
    so many requests a segment lies in one run, whose running sums serve all of it.
    The outputs [R, new, heads * d], and for every token the sums of weights and of
    weighted values in 64 bits."""
    s = Setup(S, [ctx], [new], hkv, hkv, d, 64, dtype, seed=23, spare_rows=R - 1, T=R * new)
    s.oracle_plan()
    n = ctx + new
    s.kv.table[:] = torch.from_numpy(s.table[:, :, s.rows[0]]).cuda()[:, :, None]
    b = s.plan(ctx=s.dev([ctx] * R), new=s.dev([new] * R), pages=s.dev(np.tile(s.opened, R)), rows=s.dev(np.arange(R)))
    k = torch.zeros(n, hkv * d, device="cuda")
    k[1000] = above / (4.0 * d ** 0.5)       # q . k scale = above
    v = rest(n, hkv * d).to(TDT[dtype])
    v[1000] = sink
    cache = s.cache_rows()
    cache[s.slot_rows(0, 0, 0)] = k.to(TDT[dtype])
    cache[s.slot_rows(0, 0, 1)] = v
    q = torch.full((R * new, hkv * d), 4.0, dtype=TDT[dtype], device="cuda")
    out = torch.empty_like(q)
    s.kv.attend(b, 0, q, out)
    assert s.pool.status() == S.OK
    w = torch.full((n, 1), math.exp(-above), dtype=torch.float64, device="cuda")
    w[1000] = 1
    sums = torch.cumsum(w, 0)[-new:], torch.cumsum(w * v.double(), 0)[-new:]
    s.close()
    return out.view(R, new, -1).double(), *sums


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("above", [14, 17, 18, 20])
@pytest.mark.parametrize("ctx,new,hkv,d,R", [(1 << 17, 1, 16, 16, 114), (1 << 17, 16, 4, 64, 40)])
def test_small_weights_of_a_long_context(S, dtype, above, ctx, new, hkv, d, R):
    """One key `above` nats over 131,072 others, its value zero: the result is what
    all the others add up to, e^-above each, in the decode and the chunk kernel.

    Tolerance: the result's rounding and, in the chunk kernel, the weights' (u each);
    2^-12 for fp32 arithmetic; the products, one for every 16 keys (two in the decode
    kernel), cut off at most 2^-23 of the running sum each; and the weights' own error
    below fp16's exponents, 2^-32 of the largest for each key (2^-39)."""
    out, w, want = _long_segments(S, ctx, new, hkv, d, R, dtype, above, 0.0,
                                  lambda n, c: torch.randn(n, c, device="cuda").abs())
    u, decode = U[dtype], new == 1
    tol = (2 * u + 2.0 ** -12 + ctx * 2.0 ** (-26 if decode else -27)) * want / w
    tol += 2.0 ** (-39 if decode else -32) * math.exp(above) * want
    err = (out - want / w).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunk_sum_of_small_weights_beside_a_large_one(S, dtype):
    """One key 17.4375 nats over 262,144 others, alone with a value: the result is 1
    over the sum of the weights, 0.7 % of it in weights below 2^-25 of the largest.
    Tolerance: the result's rounding and 2^-12."""
    out, w, want = _long_segments(S, 1 << 18, 16, 4, 64, 40, dtype, 17.4375, 1.0,
                                  lambda n, c: torch.zeros(n, c, device="cuda"))
    err = (out * w / want - 1).abs().max().item()
    assert err <= U[dtype] + 2.0 ** -12, err


def test_a_step_without_new_tokens(S):
    """Planned with max_new 0 (room for tokens, none in use): append and attend write nothing."""
    s = Setup(S, [4, 8], [0, 0], 2, 1, 64, 4, "f16", T=6)
    b = s.plan()
    q = s.randn(6, 128)
    out = torch.full((6, 128), 3.0, dtype=torch.float16, device="cuda")
    before = s.pool.buffer.clone()
    s.kv.append(b, 0, q, q[:, :64], q[:, 64:], q_out=out)
    s.kv.attend(b, 0, q, out)
    assert s.pool.status() == S.OK and (out == 3).all()
    assert torch.equal(s.pool.buffer.view(torch.int16), before.view(torch.int16))
    s.close()


def test_a_batch_of_another_cache_is_refused(S):
    """Two caches on one pool, planned in lock-step with different sizes: a batch's
    tensors are checked for its own T, so the other cache must not take it."""
    s = Setup(S, [4, 8], [1, 1], 2, 1, 64, 4, "f16", T=6)
    other = S.KVCache(s.pool, 1, 2, 1, 64, 4, 8)
    mine = s.plan()
    pages = s.dev([0, 1] * 2)
    theirs = other.plan(s.dev([0, 0]), s.dev([1, 1]), pages, 2, 1)
    q, out = s.randn(6, 128), torch.full((6, 128), 3.0, dtype=torch.float16, device="cuda")
    for kv, b in ((s.kv, theirs), (other, mine)):
        with pytest.raises(S.SloraError) as e:
            kv.append(b, 0, q, q[:, :64], q[:, 64:], q_out=out)
        assert e.value.code == S.ERR_INVALID
        with pytest.raises(S.SloraError) as e:
            kv.attend(b, 0, q, out)
        assert e.value.code == S.ERR_INVALID
    assert (out == 3).all()
    other.append(theirs, 0, q, q[:, :64], q[:, 64:], q_out=out)
    other.attend(theirs, 0, q, out)
    assert s.pool.status() == S.OK and (out[2:] == 3).all()
    other.close()
    s.close()


def test_plan_is_quick_at_lengths_that_are_no_batch(S):
    """New tokens far beyond T (a caller's mistake that only the device sees) are left out
    and reported without counting their tiles one by one."""
    P, R = 1024, 3
    pool = S.Pool(40, 64 * P, "f16", [(8, 8)], 1, 1, 8, device=torch.device("cuda", 0))
    kv = S.KVCache(pool, 1, 32, 1, 64, R, (1 << 30) // P)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = dev([0, 5, 77]), dev([1 << 30, (1 << 30) - 5, 1 << 29]), dev([0, 1])
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    kv.plan(dev([0]), dev([1]), dev([0, 1]), 8, 1)
    assert pool.status() == S.OK
    start.record()
    b = kv.plan(*args, 8, 1 << 30)
    end.record()
    assert pool.status() == S.ERR_INVALID
    assert not b.kv_len.any() and (b.tok_req == -1).all()
    assert start.elapsed_time(end) < 20.0        # 2^27 steps a request took a second
    kv.close()
    pool.close()


@pytest.mark.parametrize("dtype,hq,ctx,new", [("f16", 32, 0, 700), ("bf16", 31, 333, 517), ("f16", 20, 127, 900),
                                               ("bf16", 9, 5, 2000)])
def test_chunks_of_many_tiles(S, dtype, hq, ctx, new):
    """More than 64 pairs of row tiles in a request, beside requests with none and one."""
    s = Setup(S, [ctx, 40, 0], [new, 1, 3], hq, 1, 64, 4, dtype, seed=27)
    _, q, out = _fill_and_attend(S, s)
    _check_attend(s, q, out)
    s.close()


def test_overlapping_results_are_refused(S):
    """out over q (attend), q_out over q but for in place (append); slices of one product
    side by side are no overlap."""
    s = Setup(S, [4, 8, 9], [1, 1, 1], 2, 1, 64, 4, "f16")
    b, q, out = _fill_and_attend(S, s)
    w = 128
    two = torch.zeros(8, 2 * w, dtype=torch.float16, device="cuda")
    flat = torch.zeros(8 * w, dtype=torch.float16, device="cuda")
    k, v = s.randn(3, 64), s.randn(3, 64)
    rows = lambda at: flat[at: at + 3 * w].view(3, w)
    bad = [(two[:3, :w], two[:3, :w]), (two[:3, :w], two[:3, 64: 64 + w]), (two[:3, 64: 64 + w], two[:3, :w]),
           (rows(0), rows(2 * w)), (rows(3 * w - 8), rows(0)), (two[:3, w:], two[1:4, 64: 64 + w])]
    for a, o in bad:
        with pytest.raises(S.SloraError) as e:
            s.kv.attend(b, 0, a, o)
        assert e.value.code == S.ERR_INVALID
        if a.data_ptr() != o.data_ptr():
            with pytest.raises(S.SloraError) as e:
                s.kv.append(b, 0, a, k, v, q_out=o)
            assert e.value.code == S.ERR_INVALID
    good = [(two[:3, :w], two[:3, w:]), (two[:3, w:], two[:3, :w]), (two[1:4, w:], two[:3, :w]),
            (rows(0), rows(3 * w)), (rows(3 * w), rows(0)), (two[:3, :w], two[3:6, 64: 64 + w])]
    for a, o in good:
        a.copy_(q)
        s.kv.attend(b, 0, a, o)
        assert torch.equal(o, out[:3, :w])
    for a, o in good + [(q, None)]:
        s.kv.append(b, 0, a, k, v, q_out=o)
    assert s.pool.status() == S.OK
    s.close()


def test_more_rows_than_31_bits_count_are_refused(S):
    """32,768 tokens of 65,536 query heads (refused before any pointer is used)."""
    T, heads = 1 << 15, 1 << 16
    pool = S.Pool(40, 64, "f16", [(8, 8)], 1, 1, T, device=torch.device("cuda", 0))
    kv = S.KVCache(pool, 1, heads, 1, 16, 2, T // 4)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    b = kv.plan(z, z, None, T, T)
    with pytest.raises(S.SloraError) as e:
        S.slora_kv_attend(kv.handle, b.raw, 0, pool.buffer.data_ptr(), heads * 16, z.data_ptr(), heads * 16, 1.0)
    assert e.value.code == S.ERR_INVALID and "2^31" in str(e.value)
    assert pool.status() == S.OK
    kv.close()
    pool.close()


def test_cache_memory_belongs_to_the_compute_stream(S, monkeypatch):
    """The table and the batch arrays are cleared on the pool's compute stream, so that
    is the stream they are allocated for, whichever is current."""
    stream = torch.cuda.Stream()
    pool = S.Pool(8, 256, "f16", [(8, 8)], 1, 1, 4, device=torch.device("cuda", 0), compute_stream=stream)
    seen, real = [], torch.empty

    def empty(*a, **kw):
        seen.append(torch.cuda.current_stream())
        return real(*a, **kw)

    monkeypatch.setattr(torch, "empty", empty)
    kv = S.KVCache(pool, 1, 2, 1, 64, 2, 3)
    assert len(seen) == 2 and all(x == stream for x in seen)
    assert torch.cuda.current_stream() != stream
    stream.synchronize()
    assert (kv.table == -1).all() and not kv.arrays.any()
    kv.close()
    pool.close()


def test_batches_of_many_sizes_leave_nothing_behind(S):
    """A server's (R, T) changes every step: the cache keeps no views of batches, and a
    batch's are right when they are asked for."""
    s = Setup(S, [3, 0, 9], [1, 5, 2], 2, 1, 16, 4, "f16", layers=3, T=40)
    size = lambda: sum(len(x) for x in vars(s.kv).values() if isinstance(x, (dict, list)))
    before = size()
    for T in range(8, 41):
        b = s.plan(T=T)
        s.T = T
        want = s.oracle_plan()
    assert size() == before
    for k, w in want.items():
        assert np.array_equal(getattr(b, k).cpu().numpy(), w), k
    assert s.pool.status() == S.OK
    s.close()


def test_debug_build_catches_planted_indices():
    """The SLORA_DEBUG build, in a process of its own: tests/debug_kv_check.py."""
    from lora_adapters_gb300 import build

    build.build(debug=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-m", "tests.debug_kv_check"], cwd=root, env=dict(os.environ, SLORA_DEBUG="1"),
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "debug build OK" in res.stdout
