"""Numerics of key-value caches held in 4 bits on the GPU: values, scales and scores at the ends of
their ranges, groups that are not finite, heads whose last group is half full.  Tolerances as in
tests/test_gpu_kv_q4.py unless a test says its own.
"""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from oracle import kv_q4 as oq4
from tests.test_gpu_kv_q4 import S, TDT, U, Setup, _attend, _check, f64  # noqa: F401

pytestmark = pytest.mark.gpu


def _store(s, r, j, k, M):
    """Codes k [n, heads, 32 ng] and scales M [n, heads, ng] as request r's keys (j 0) or values."""
    s.row_view()[s.at(r, 0, j)] = torch.from_numpy(oq4.pack(k, M, s.dtype, j == 1)).cuda()


def _random(s, n, M):
    """Codes for n tokens, and scales of random sign and at most five bits near M [n, heads, ng]."""
    k = s.rng.integers(-7, 9, (n, s.hkv, 32 * oq4.groups(s.d)))
    round_ = np.vectorize(lambda m: oq4.scale(m, s.dtype), otypes=[np.float64])
    return k, round_(M * s.rng.choice([-1.0, 1.0], (n, s.hkv, oq4.groups(s.d))))


def _leave_nans_in_shared_memory(S):  # noqa: F811
    """A chunk call over queries and a pool whose bits are all ones: they fill every SM's shared memory."""
    s = Setup(S, [0], [2048], 8, 8, 128, 1024, "f16")
    b = s.plan()
    q = torch.full((s.T, 8 * 128), -1, dtype=torch.int16, device="cuda").view(torch.float16)
    s.kv.attend(b, 0, q, torch.empty_like(q))
    torch.cuda.synchronize()
    return s                                       # (kept: freeing its pool would run other kernels)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rot", ["half", "interleaved", "none"])
@pytest.mark.parametrize("hkv,d", [(3, 16), (5, 48), (3, 80), (2, 112), (1, 144), (2, 176), (1, 208), (3, 240)])
def test_normed_heads_whose_last_group_is_half_full(S, dtype, rot, hkv, d):  # noqa: F811
    """The bytes of a normed append are the oracle's, whatever lay in shared memory before it."""
    s = Setup(S, [7], [40], 2 * hkv, hkv, d, oq4.row_bytes(hkv, d) * 2, dtype)
    freq = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    rot_dim = 0 if rot == "none" else d
    s.kv.set_rotary(rot_dim, freq, interleaved=rot == "interleaved")
    b = s.plan()
    want = s.oracle_plan()
    q, k, v = s.randn(s.T, 2 * hkv * d), s.randn(s.T, hkv * d), s.randn(s.T, hkv * d)
    w = s.randn(d, scale=0.3) + 1
    q_out = torch.empty_like(q)
    view = s.row_view()
    other = _leave_nans_in_shared_memory(S)
    s.kv.append(b, 0, q, k, v, q_out=q_out, q_weight=w, k_weight=w, eps=1e-5)
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    used = 18 * oq4.groups(d) * hkv
    for t in range(s.T):
        y = okv.norm_rotate(f64(k[t]).reshape(hkv, d), f64(w), 1e-5, int(want["tok_pos"][t]), freq, rot_dim,
                            rot == "interleaved", 1.0)
        for j, x in ((0, y), (1, f64(v[t]).reshape(hkv, d))):
            slot = int(want["slots"][0, j, t])
            row = oq4.pack(*(z[None] for z in oq4.quantise(x, dtype)), dtype, j == 1)[0]
            assert np.array_equal(view[slot // s.P, slot % s.P].cpu().numpy()[:used], row[:used]), (t, j)
    other.close()
    s.close()


SHAPES = [   # hq, hkv, d: tiles of two, four and eight rows, every number of groups
    (4, 4, 128), (3, 3, 96), (2, 2, 160), (6, 3, 192), (1, 1, 224), (2, 2, 256),
    (8, 2, 128), (4, 4, 64), (12, 3, 96), (8, 1, 128), (8, 1, 256), (5, 1, 192), (24, 3, 64), (2, 2, 32)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("new", [1, 60])
def test_a_value_group_that_is_not_finite_leaves_the_others(S, dtype, hq, hkv, d, new):  # noqa: F811
    """One token's group of one head's values is NaN: so is that group of the results of that head's
    queries, and every other element is what it would be without it."""
    s = Setup(S, [40, 3000, 90], [new, new, 1], hq, hkv, d, oq4.row_bytes(hkv, d) * 2, dtype, seed=14)
    s.oracle_plan()
    held, ng = s.fill(), oq4.groups(d)
    where = {}                                     # request: (token, head, group)
    for r, (p, h, g) in {0: (0, hkv - 1, 0), 1: (1500, 0, ng - 1), 2: (90, hkv - 1, ng // 2)}.items():
        page, at = (int(x[p]) for x in s.at(r, 0, 1))
        scale = s.row_view()[page, at, 16 * ng * hkv: 18 * ng * hkv].view(torch.int16)
        scale[h * ng + g] = 0x7fff
        held[r][1][p, h, 32 * g: 32 * g + 32] = 0.0
        where[r] = (h, g)
    b = s.plan()
    q, out = s.randn(s.T, hq * d, scale=0.01), torch.empty(s.T, hq * d + 8, dtype=TDT[dtype], device="cuda")
    out[:, hq * d:] = 3.0
    s.kv.attend(b, 0, q, out[:, : hq * d])
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    t0, group = 0, hq // hkv
    for r, n in enumerate(s.new):
        h, g = where[r]
        bad = torch.zeros(n, hkv, group, d, dtype=torch.bool, device="cuda")
        bad[:, h, :, 32 * g: 32 * g + 32] = True
        got = out[t0: t0 + n, : hq * d].unflatten(1, (hkv, group, d))
        assert torch.equal(got.isnan(), bad), r
        # (what the group would be without its NaN token: the oracle's, to compare the rest)
        want = okv.attend(f64(q[t0: t0 + n]).reshape(n, hq, d), *held[r], s.ctx[r], d ** -0.5, 0.0)
        got[bad] = torch.from_numpy(want).to(got).unflatten(1, (hkv, group))[bad]
        t0 += n
    _check(s, held, q, out)
    s.close()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_zeros_beside_large_elements(S, dtype, hq, hkv, d):  # noqa: F811
    """Elements that are zero in every token, beside elements as large as M, with weights that
    differ: zeros come out.  Their codes are 7, so a result is sum(w 7) - 7 sum(w) over the products w
    of a weight and M / 8, the same w in both but for an fp16 cache's second part, 2^-21 of it: the
    sums' own rounding is left.  Of it, relative to the largest sum: a unit's product 2^-20 (at
    most 32 products added up and cut off), the sum over at most 13 units 13 2^-24, a lane's sum 28
    2^-24, the lanes' and the rest 8 2^-24.  In all below 2^-17, times 7 / 8 of the largest M."""
    s = Setup(S, [3, 33, 200], [1, 1, 1], hq, hkv, d, oq4.row_bytes(hkv, d) * 2, dtype, seed=15)
    s.oracle_plan()
    held, ng = s.fill(), oq4.groups(d)
    top = []
    for r in range(3):
        n = s.ctx[r] + 1
        k, M = _random(s, n, s.rng.uniform(0.5, 1.0, (n, hkv, ng)))
        k[:, :, ::2] = 0
        _store(s, r, 1, k, M)
        held[r][1] = oq4.values(k, M, d)
        top.append(np.abs(M).max())
    b, q, out = _attend(s, held)
    got = f64(out[:, : hq * d]).reshape(3, hq, d)
    for r in range(3):
        assert np.abs(got[r, :, ::2]).max() <= 7 / 8 * 2.0 ** -17 * top[r], (r, np.abs(got[r, :, ::2]).max())
        assert np.abs(got[r, :, 1::2]).max() > 0.01
    s.close()


@pytest.mark.parametrize("dtype,low,high", [("bf16", -99, -93), ("bf16", -97, -96), ("bf16", 124, 127), ("f16", -21, -17),
                                            ("f16", 14, 15)])
@pytest.mark.parametrize("hq,hkv,new,d", [(4, 4, 1, 128), (8, 1, 1, 128), (8, 2, 1, 96), (4, 2, 60, 128), (2, 2, 2, 256)])
def test_values_at_the_ends_of_the_range(S, dtype, low, high, hq, hkv, new, d):  # noqa: F811
    """Caches whose values are all very small, or all very large, against their largest.  (fp16
    results below 2^-14 are multiples of 2^-24: the rounding of one is off by up to 2^-25, where
    2^-11 of the result is less.)"""
    s = Setup(S, [300, 20], [new, new], hq, hkv, d, oq4.row_bytes(hkv, d) * 2, dtype, seed=8)
    s.oracle_plan()
    held = s.fill()
    for r in range(2):
        n = s.ctx[r] + s.new[r]
        k, M = _random(s, n, 2.0 ** s.rng.uniform(low, high, (n, hkv, oq4.groups(d))))
        _store(s, r, 1, k, M)
        held[r][1] = oq4.values(k, M, d)
    b = s.plan()
    q, out = s.randn(s.T, hq * d, scale=2.0), torch.empty(s.T, hq * d, dtype=TDT[dtype], device="cuda")
    s.kv.attend(b, 0, q, out)
    assert s.pool.status() == S.OK
    t0, u = 0, U[dtype]
    for r, n in enumerate(s.new):
        want = okv.attend(f64(q[t0: t0 + n]).reshape(n, hq, d), *held[r], s.ctx[r], d ** -0.5, 0.0)
        vmax = np.repeat(np.abs(held[r][1]).max((0, 2)), hq // hkv)[None, :, None]
        tol = np.maximum(u * np.abs(want), 2.0 ** -25 if dtype == "f16" else 0.0) + (
            2.0 ** -12 + (u if new * hq // hkv > 8 else 0.0)) * vmax
        err = np.abs(f64(out[t0: t0 + n]).reshape(n, hq, d) - want)
        assert (err <= tol).all(), (r, float((err / tol).max()))
        t0 += n
    s.close()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,new,d", [(4, 4, 1, 128), (8, 2, 1, 64), (8, 1, 1, 256), (4, 2, 60, 128)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_scales_of_scores_that_are_next_to_nothing(S, dtype, hq, hkv, new, d, softcap):  # noqa: F811
    """A scale so small that every score is zero, and queries of zeros: equal weights for the keys
    that a row may see, none for the others."""
    s = Setup(S, [5, 700], [new, new], hq, hkv, d, oq4.row_bytes(hkv, d) * 2, dtype, seed=16)
    s.oracle_plan()
    held = s.fill()
    b = s.plan()
    for q in (s.randn(s.T, hq * d), torch.zeros(s.T, hq * d, dtype=TDT[dtype], device="cuda")):
        for scale in (1e-20, 1e-38):
            out = torch.full((s.T, hq * d + 8), 3.0, dtype=TDT[dtype], device="cuda")
            s.kv.attend(b, 0, q, out[:, : hq * d], scale=scale, softcap=softcap)
            assert s.pool.status() == S.OK
            _check(s, held, q, out, softcap, scale)
    s.close()


@pytest.mark.parametrize("hq,hkv,new,d", [(4, 4, 1, 128), (8, 2, 1, 64), (8, 1, 1, 256)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("zero_keys", [False, True])
def test_scores_near_the_largest_number(S, hq, hkv, new, d, softcap, zero_keys):  # noqa: F811
    """Queries whose scores reach 2^122: the largest one has all the weight (or what the cap leaves
    it); keys of zeros have scores of zero all the same."""
    dtype = "bf16"
    s = Setup(S, [5, 700], [new, new], hq, hkv, d, oq4.row_bytes(hkv, d) * 2, dtype, seed=17)
    s.oracle_plan()
    held = s.fill()
    for r in range(2):
        n = s.ctx[r] + s.new[r]
        k, M = _random(s, n, s.rng.uniform(0.25, 1.0, (n, hkv, oq4.groups(d))))
        if zero_keys:
            k[:], M[:] = 0, 0.0
        _store(s, r, 0, k, M)
        held[r][0] = oq4.values(k, M, d)
    b = s.plan()
    q = torch.zeros(s.T, hq, d, dtype=TDT[dtype], device="cuda")
    q[:, :, 37 % d] = 2.0 ** 125
    q[:, hq // 2:, 37 % d] *= -1
    q, out = q.view(s.T, hq * d), torch.full((s.T, hq * d + 8), 3.0, dtype=TDT[dtype], device="cuda")
    s.kv.attend(b, 0, q, out[:, : hq * d], softcap=softcap)
    assert s.pool.status() == S.OK
    _check(s, held, q, out, softcap)
    s.close()


@pytest.mark.parametrize("hq,hkv,new,d", [(4, 4, 1, 128), (4, 4, 1, 160), (2, 2, 1, 256), (8, 1, 1, 256), (4, 2, 60, 128)])
def test_keys_of_the_largest_numbers(S, hq, hkv, new, d):  # noqa: F811
    """Keys as large as a bf16 cache holds, all of one sign, against queries of one sign that
    bring their products back: scores of ordinary size."""
    s = Setup(S, [5, 300], [new, new], hq, hkv, d, oq4.row_bytes(hkv, d) * 2, "bf16", seed=18)
    s.oracle_plan()
    held = s.fill()
    for r in range(2):
        n = s.ctx[r] + s.new[r]
        k = s.rng.integers(7, 9, (n, hkv, 32 * oq4.groups(d)))
        M = np.full((n, hkv, oq4.groups(d)), oq4.LARGEST["bf16"])
        k[::3] = s.rng.integers(-7, 9, k[::3].shape)
        _store(s, r, 0, k, M)
        held[r][0] = oq4.values(k, M, d)
    b = s.plan()
    q = torch.full((s.T, hq * d), 1.9921875 * 2.0 ** -100, dtype=torch.bfloat16, device="cuda")
    out = torch.full((s.T, hq * d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    scale = float(np.float32(8.0 / (d * 2.0 ** 29)))
    s.kv.attend(b, 0, q, out[:, : hq * d], scale=scale)
    assert s.pool.status() == S.OK
    _check(s, held, q, out, scale=scale)
    s.close()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 80, 96, 112, 128])
def test_chunks_of_every_head_size_and_cap(S, dtype, d):  # noqa: F811
    s = Setup(S, [70, 3], [20, 11], 4, 2, d, oq4.row_bytes(2, d) * 2, dtype, seed=19)
    s.oracle_plan()
    held = s.fill()
    for softcap in (0.0, 20.0, 100.0):
        _attend(s, held, softcap=softcap)
    s.close()


OUTLIERS = {"none": 1.0, "64": 64.0, "1000": 1000.0, "infinite": float("inf")}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rot", ["half", "interleaved", "part"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d", [64, 96, 128, 240])
@pytest.mark.parametrize("size", OUTLIERS)
def test_keys_with_outliers(S, dtype, rot, norm, d, size):  # noqa: F811
    """Heads with an element far above the rest: the bytes are the oracle's in every group."""
    hkv = 3
    s = Setup(S, [90], [32], hkv, hkv, d, oq4.row_bytes(hkv, d) * 2, dtype, seed=21)
    freq = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    rot_dim = 16 if rot == "part" else d
    s.kv.set_rotary(rot_dim, freq, interleaved=rot == "interleaved")
    b = s.plan()
    want = s.oracle_plan()
    k = s.randn(s.T, hkv * d)
    k[:, 5::d] *= OUTLIERS[size]
    w = s.randn(d, scale=0.3) + 1 if norm else None
    s.kv.append(b, 0, k.clone(), k, k, q_out=torch.empty_like(k), q_weight=w, k_weight=w, eps=1e-5)
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    used = 18 * oq4.groups(d) * hkv
    for t in range(s.T):
        with np.errstate(invalid="ignore"):
            y = okv.norm_rotate(f64(k[t]).reshape(hkv, d), f64(w) if norm else None, 1e-5, int(want["tok_pos"][t]), freq,
                                rot_dim, rot == "interleaved", 1.0)
        slot = int(want["slots"][0, 0, t])
        got = s.row_view()[slot // s.P, slot % s.P].cpu().numpy()[None]
        codes, M = oq4.quantise(y, dtype)
        row = oq4.pack(codes[None], M[None], dtype, False)
        held, expect = oq4.unpack(got, hkv, d, dtype, False), oq4.unpack(row, hkv, d, dtype, False)
        assert np.array_equal(held, expect, equal_nan=True), t
        if not np.isnan(M).any():                  # (the codes of a group that is NaN are not defined)
            assert np.array_equal(got[0, :used], row[0, :used]), t
    s.close()


def test_a_pair_of_which_one_leaves_the_range(S):  # noqa: F811
    """Turned by an eighth of a circle and a little, a pair of the largest keys becomes one past fp32's
    range, whose group is NaN, and a small one, of which fp32 has no bit: its group's bytes
    are the oracle's."""
    d, T = 64, 40
    s = Setup(S, [0], [T], 1, 1, d, 512, "bf16", seed=22)
    off = np.logspace(-10, -8, T)
    freq = [0.0] * (d // 2)
    k = s.randn(T, d).double() * 3e29
    k[:, 0] = k[:, 32] = 3.3e38
    k = k.to(torch.bfloat16)
    for t in range(1, T):                          # (one token a call: every one has its own angle)
        s.ctx, s.new, s.T = [t], [1], 1
        freq[0] = (np.pi / 4 + off[t]) / t
        s.kv.set_rotary(d, freq)
        block = t // s.P                           # K's page and V's
        s.kv.table[0, :, :, block] = s.dev([2 * block, 2 * block + 1])[:, None]
        opens = s.dev([2 * block, 2 * block + 1]) if t % s.P == 0 else None
        b = s.kv.plan(s.dev([t]), s.dev([1]), opens, 1, 1, rows=s.dev(s.rows))
        s.kv.append(b, 0, k[t: t + 1].clone(), k[t: t + 1], k[t: t + 1])
        torch.cuda.synchronize()
        assert s.pool.status() == S.OK
        y = okv.norm_rotate(f64(k[t]).reshape(1, d), None, 0.0, t, freq, d, False, 1.0)
        assert abs(y[0, 0]) < 1e31 and y[0, 32] > 3.41e38
        out = torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
        s.kv.read(0, s.dev(s.rows), s.dev([t]), out)
        assert out[0, 32:].isnan().all()
        assert np.array_equal(f64(out)[0, :32], oq4.values(*oq4.quantise(y, "bf16"), d)[0, :32]), t
    s.close()



@pytest.mark.parametrize("norm", [False, True])
def test_outliers_do_not_slow_the_append(S, norm):  # noqa: F811
    """An element far above the rest of its head, or an infinite one, leaves few elements of the other
    groups near a border: the append takes about as long as without it (it was 4 to 11 times as long)."""
    hkv, d, T = 32, 128, 512
    s = Setup(S, [90], [T], hkv, hkv, d, 4096, "f16")
    s.kv.set_rotary(d, [10000.0 ** (-2 * i / d) for i in range(d // 2)])
    b = s.plan()
    plain, w = s.randn(T, hkv * d), s.randn(d, scale=0.3) + 1 if norm else None
    out, took = torch.empty_like(plain), {}
    for size in OUTLIERS:
        k = plain.clone()
        k[:, 5::d] *= OUTLIERS[size]
        times = []
        for _ in range(7):
            ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            with torch.cuda.stream(s.pool.compute_stream):
                ev[0].record()
                for _ in range(8):
                    s.kv.append(b, 0, plain, k, k, q_out=out, q_weight=w, k_weight=w)
                ev[1].record()
            torch.cuda.synchronize()
            times.append(ev[0].elapsed_time(ev[1]) / 8)
        took[size] = min(times)
    assert max(took.values()) < 2.5 * took["none"], took
    s.close()
