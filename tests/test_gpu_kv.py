"""The paged key-value cache operators on the GPU against the fp64 oracle:
slora_kv_plan, slora_kv_append, slora_kv_attend.

Tolerances.  u is the largest relative error of one rounding to the storage
type (fp16 2^-11, bf16 2^-8).
 - append: one rounding of values computed in fp32.  An element is a sum of
   two products of normed values (|x| below about 6 times its weight), cosine
   and sine good to 2^-22 of a unit: |err| <= u |y| + 2^-18 max|pair|.
 - attend: one rounding of the result, u |o|; scores of at most 256 fp32
   products leave a relative error below 2^-12 in a weight; and the weights of
   requests with more than 8 rows (new tokens times query heads a key head)
   may themselves be rounded to the storage type, where they add at most u
   times the largest |v| of the request's head (with up to 8 rows they keep
   twice the 16 bits).
"""
import numpy as np
import pytest
import torch

from oracle import kv as okv

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TDT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def S():
    from lora_adapters_gb300 import build, slora

    build.build()
    slora.lib()
    return slora


def f64(t):
    return t.detach().cpu().double().numpy()


class Setup:
    """A pool whose every slot holds NaN except the tokens a request stores,
    and a cache with the requests' context blocks in its table."""

    def __init__(self, S, ctx, new, hq, hkv, d, P, dtype, layers=1, seed=0, spare_rows=2, T=None, first_page=0,
                 spread=2.0):
        self.S = S
        rng = np.random.default_rng(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx, self.new, self.P, self.L, self.d, self.hq, self.hkv = ctx, new, P, layers, d, hq, hkv
        self.dtype, R = dtype, len(ctx)
        self.T = sum(new) if T is None else T
        blocks = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        n_blocks = sum(blocks)
        self.num_pages = first_page + n_blocks * 2 * layers + 3
        order = rng.permutation(n_blocks * 2 * layers + 3)[: n_blocks * 2 * layers] + first_page
        self.pages = order.reshape(n_blocks, layers, 2)
        self.H = hkv * d * P
        self.pool = S.Pool(self.num_pages, self.H, dtype, [(8, 8)], 1, 1, max(self.T, 1), device=torch.device("cuda", 0))
        self.pool.buffer[first_page:].fill_(float("nan"))
        max_rows = R + spare_rows
        self.rows = rng.permutation(max_rows)[:R].astype(np.int32)
        self.max_blocks = max(blocks + [1])
        self.kv = S.KVCache(self.pool, layers, hq, hkv, d, max(1, max_rows), self.max_blocks)
        self.table = np.full((layers, 2, max_rows, self.max_blocks), -1, np.int32)
        opened, b = [], 0
        for r in range(R):
            for i in range(blocks[r]):
                if i >= -(-ctx[r] // P):
                    opened.append(self.pages[b])
                else:
                    self.table[:, :, self.rows[r], i] = self.pages[b]
                b += 1
        self.kv.table.copy_(torch.from_numpy(self.table))
        self.opened = np.array(opened, np.int32).reshape(-1)

    def dev(self, x):
        return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()

    def plan(self, **kw):
        args = dict(ctx=self.dev(self.ctx), new=self.dev(self.new), pages=self.dev(self.opened), T=self.T,
                    max_new=max(self.new + [0]), rows=self.dev(self.rows))
        args.update(kw)
        return self.kv.plan(**args)

    def oracle_plan(self):
        return okv.plan(self.table, self.rows, self.ctx, self.new, self.opened, self.T, self.P, self.num_pages)

    def randn(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(TDT[self.dtype])

    def slot_rows(self, r, layer, kv):
        """Pool rows of the tokens request r holds after the step (from the oracle's table)."""
        p = np.arange(self.ctx[r] + self.new[r])
        return torch.from_numpy(self.table[layer, kv, self.rows[r], p // self.P].astype(np.int64) * self.P
                                + p % self.P).cuda()

    def cache_rows(self):
        return self.pool.buffer.view(-1, self.hkv * self.d)

    def close(self):
        self.kv.close()
        self.pool.close()


PLANS = {
    # (ctx, new, P, layers, T)
    "decode": ([5, 0, 17, 640, 1], [1, 1, 1, 1, 1], 1, 3, None),
    "decode_blocks": ([5, 0, 16, 639, 15, 31], [1, 1, 1, 1, 1, 1], 16, 2, None),
    "chunks": ([0, 0, 7, 100, 33], [300, 1, 0, 57, 129], 5, 2, None),
    "room_to_spare": ([0, 9], [3, 1], 4, 1, 70),
    "none_new": ([4, 8], [0, 0], 4, 1, 6),
    "no_requests": ([], [], 2, 1, 3),
    "many": (list(range(700)), [i % 3 for i in range(700)], 3, 33, None),
}


@pytest.mark.parametrize("name", PLANS)
def test_plan_matches_oracle(S, name):
    ctx, new, P, layers, T = PLANS[name]
    s = Setup(S, ctx, new, 2, 1, 16, P, "f16", layers=layers, T=T)
    for _ in range(2):                       # planning the same step again changes nothing
        b = s.plan()
        torch.cuda.synchronize()
        want = s.oracle_plan()
        for k, w in want.items():
            assert np.array_equal(getattr(b, k).cpu().numpy(), w), k
        assert np.array_equal(s.kv.table.cpu().numpy()[:, :, : s.table.shape[2]], s.table)
    assert s.pool.status() == S.OK
    s.close()


def test_plan_identity_rows_and_growth(S):
    """A request grown over several steps holds the blocks each step opened."""
    s = Setup(S, [0, 0], [7, 2], 2, 1, 16, 4, "f16", layers=2, T=16, spare_rows=0)
    s.rows = np.array([0, 1], np.int32)
    table = np.full_like(s.table, -1)
    ctx, nxt = np.zeros(2, np.int32), 0
    for new in ([3, 1], [1, 0], [2, 1], [1, 0]):
        new = np.array(new, np.int32)
        opened = sum(-(-(c + n) // 4) - -(-c // 4) for c, n in zip(ctx, new))
        pages = np.arange(nxt, nxt + opened * 4, dtype=np.int32) % s.num_pages
        nxt += opened * 4
        want = okv.plan(table, [0, 1], ctx.tolist(), new.tolist(), pages, 16, 4, s.num_pages)
        b = s.kv.plan(s.dev(ctx), s.dev(new), s.dev(pages), 16, 3)
        assert np.array_equal(b.slots.cpu().numpy(), want["slots"])
        assert np.array_equal(s.kv.table.cpu().numpy(), table)
        ctx = ctx + new
    assert s.pool.status() == S.OK
    s.close()


def test_plan_reports_bad_requests_and_leaves_them_out(S):
    def fresh():
        return Setup(S, [4, 6, 2], [2, 1, 3], 2, 1, 16, 2, "f16", layers=1)

    cases = {
        "negative ctx": dict(ctx=[4, -1, 2]),
        "negative new": dict(new=[2, -1, 3]),
        "row outside": dict(rows=[0, 99, 1]),
        "too long for a row": dict(ctx=[4, 10 ** 6, 2]),
        "more than max_new": dict(new=[2, 4, 3], max_new=3),
    }
    for name, change in cases.items():
        s = fresh()
        s.rows = np.array([0, 1, 2], np.int32)
        s.kv.table.zero_()
        kw = {k: (v if k == "max_new" else s.dev(v)) for k, v in change.items()}
        b = s.plan(**({"rows": s.dev(s.rows)} | kw), T=s.T) if "T" not in kw else s.plan(**kw)
        assert s.pool.status() == S.ERR_INVALID, name
        assert b.kv_len.cpu().tolist()[1] == 0, name
        assert b.kv_len.cpu().tolist()[0] == 6 and b.kv_len.cpu().tolist()[2] == 5, name
        assert b.q_start.cpu().tolist() == [0, 2, 2, 5], name
        assert s.pool.status() == S.OK
        s.close()
    for name, change in {"tokens beyond T": dict(T=5), "blocks beyond pages": dict(pages=[])}.items():
        s = fresh()
        before = s.kv.table.clone()
        kw = {k: (v if k == "T" else s.dev(v)) for k, v in change.items()}
        b = s.plan(**kw)
        assert s.pool.status() == S.ERR_INVALID, name
        assert not b.kv_len.any() and not b.q_start.any() and (b.tok_req == -1).all() and (b.slots == -1).all(), name
        assert torch.equal(s.kv.table, before)
        s.close()
    # a page outside the pool: its entry is -1 and its tokens have no slot
    s = fresh()
    pages = s.opened.copy()
    pages[0], pages[1] = s.num_pages, -5
    b = s.plan(pages=s.dev(pages))
    assert s.pool.status() == S.ERR_INVALID
    assert (b.slots.cpu().numpy() == -1).sum() == 4       # two tokens, K and V
    s.close()


ROT = {   # rot_dim, interleaved, norm, mscale, factor
    "half": (0, False, False, 1.0, 1.0),
    "half_norm": (0, False, True, 1.0, 1.0),
    "interleaved": (0, True, False, 1.0, 1.0),
    "interleaved_norm_scaled": (0, True, True, 1.25, 8.0),
    "part": (32, False, True, 1.0, 1.0),
    "part_interleaved": (16, True, False, 0.5, 1.0),
    "norm_only": (-1, False, True, 1.0, 1.0),
    "copy": (-1, False, False, 1.0, 1.0),
}


@pytest.mark.parametrize("rot", ROT)
@pytest.mark.parametrize("dtype,hq,hkv,d,P", [("f16", 4, 4, 64, 1), ("bf16", 10, 2, 128, 5), ("f16", 3, 1, 80, 2),
                                               ("bf16", 2, 1, 256, 3), ("f16", 7, 7, 16, 1), ("bf16", 4, 2, 96, 4)])
def test_append_matches_oracle(S, rot, dtype, hq, hkv, d, P):
    rot_dim, inter, norm, mscale, factor = ROT[rot]
    rot_dim = d if rot_dim == 0 else max(0, min(rot_dim, d))
    ctx, new, layers = [0, 1, 131071, 40], [9, 1, 2, 0], 2
    s = Setup(S, ctx, new, hq, hkv, d, P, dtype, layers=layers, T=14)
    freq = [10000.0 ** (-2 * i / max(rot_dim, 1)) / factor for i in range(rot_dim // 2)]
    s.kv.set_rotary(rot_dim, freq, interleaved=inter, mscale=mscale)
    b = s.plan()
    want = s.oracle_plan()
    T, layer = s.T, 1
    qkv = s.randn(T, (hq + 2 * hkv) * d + 8)
    q, k, v = qkv[:, : hq * d], qkv[:, hq * d: (hq + hkv) * d], qkv[:, (hq + hkv) * d: (hq + 2 * hkv) * d]
    qw, kw = (s.randn(d, scale=0.3) + 1, s.randn(d, scale=0.3) + 1) if norm else (None, None)
    q_out = torch.full((T, hq * d + 16), 7.0, dtype=TDT[dtype], device="cuda")
    before = s.pool.buffer.clone()
    s.kv.append(b, layer, q, k, v, q_out=q_out[:, : hq * d], q_weight=qw, k_weight=kw, eps=1e-5)
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    cache, was = s.cache_rows(), before.view(-1, hkv * d)
    touched = torch.zeros(cache.shape[0], dtype=torch.bool, device="cuda")
    n_tok = sum(new)
    for t in range(n_tok):
        pos = int(want["tok_pos"][t])
        for x, w, heads, got in ((q, qw, hq, q_out[t, : hq * d]),
                                 (k, kw, hkv, cache[int(want["slots"][layer, 0, t])])):
            xv = f64(x[t]).reshape(heads, d)
            y = okv.norm_rotate(xv, f64(w) if norm else None, 1e-5, pos, freq, rot_dim, inter, mscale)
            big = max(1.0, np.abs(y).max())
            err = np.abs(f64(got).reshape(heads, d) - y)
            assert (err <= U[dtype] * np.abs(y) + 2.0 ** -18 * big).all(), (t, err.max())
        slot_k, slot_v = int(want["slots"][layer, 0, t]), int(want["slots"][layer, 1, t])
        assert torch.equal(cache[slot_v], v[t])
        touched[[slot_k, slot_v]] = True
    # nothing else was written: other slots, the padding tokens and the columns past the heads
    same = cache.view(torch.int16) == was.view(torch.int16)
    assert same[~touched].all()
    assert (q_out[n_tok:] == 7).all() and (q_out[:, hq * d:] == 7).all()
    # in place gives the same bits
    qi = qkv.clone()
    s.kv.append(b, layer, qi[:, : hq * d], k, v, q_weight=qw, k_weight=kw, eps=1e-5)
    assert torch.equal(qi[:n_tok, : hq * d], q_out[:n_tok, : hq * d])
    assert torch.equal(qi[n_tok:], qkv[n_tok:])
    s.close()


def _fill_and_attend(S, s, softcap=0.0, scale=None, layer=0, graph=False):
    b = s.plan()
    s.oracle_plan()
    hq, hkv, d, T = s.hq, s.hkv, s.d, s.T
    cache = s.cache_rows()
    for r in range(len(s.ctx)):
        n = s.ctx[r] + s.new[r]
        if n:
            cache[s.slot_rows(r, layer, 0)] = s.randn(n, hkv * d)
            cache[s.slot_rows(r, layer, 1)] = s.randn(n, hkv * d)
    q = s.randn(T, hq * d + 24, scale=2.0)[:, 8: 8 + hq * d]
    out = torch.full((T, hq * d + 8), 3.0, dtype=TDT[s.dtype], device="cuda")
    s.kv.attend(b, layer, q, out[:, : hq * d], scale=scale, softcap=softcap)
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    return b, q, out


def _check_attend(s, q, out, softcap=0.0, scale=None, layer=0, requests=None):
    hq, hkv, d = s.hq, s.hkv, s.d
    scale = d ** -0.5 if scale is None else scale
    cache = s.cache_rows()
    decode = max(s.new + [0]) * (s.hq // s.hkv) <= 8
    t0 = 0
    for r, (c, n) in enumerate(zip(s.ctx, s.new)):
        if n and (requests is None or r in requests):
            keys = f64(cache[s.slot_rows(r, layer, 0)]).reshape(-1, hkv, d)
            vals = f64(cache[s.slot_rows(r, layer, 1)]).reshape(-1, hkv, d)
            want = okv.attend(f64(q[t0: t0 + n]).reshape(n, hq, d), keys, vals, c, scale, softcap)
            got = f64(out[t0: t0 + n, : hq * d]).reshape(n, hq, d)
            vmax = np.repeat(np.abs(vals).max((0, 2)), hq // hkv)[None, :, None]
            u = U[s.dtype]
            tol = u * np.abs(want) + (2.0 ** -12 + (0.0 if decode else u)) * vmax
            err = np.abs(got - want)
            assert (err <= tol).all(), (r, c, n, float((err / tol).max()))
        t0 += n
    assert (out[t0:] == 3).all() and (out[:, hq * d:] == 3).all()


ATTEND = {
    # ctx, new, hq, hkv, d, P, dtype, softcap
    "one_token": ([0], [1], 4, 4, 64, 1, "f16", 0.0),
    "one_key_head": ([777], [1], 8, 1, 128, 4, "bf16", 0.0),
    "decode": ([0, 1, 15, 16, 17, 63, 64, 200, 1000], [1] * 9, 8, 8, 128, 1, "f16", 0.0),
    "decode_group5": ([0, 3, 130, 511, 900], [1] * 5, 20, 4, 128, 5, "bf16", 0.0),
    "decode_group16": ([40, 333], [1, 1], 32, 2, 64, 8, "f16", 0.0),
    "decode_group24": ([40, 333], [1, 1], 24, 1, 64, 8, "f16", 30.0),
    "decode_d80": ([12, 90, 257], [1] * 3, 6, 3, 80, 2, "f16", 0.0),
    "decode_d256": ([12, 90, 257], [1] * 3, 4, 2, 256, 3, "bf16", 20.0),
    "decode_d16": ([100, 7], [1, 1], 3, 3, 16, 7, "f16", 0.0),
    "decode_heads20": ([100, 7, 64], [1] * 3, 20, 20, 64, 1, "bf16", 0.0),
    "some_none": ([5, 80, 0, 0, 31], [1, 0, 0, 1, 1], 8, 2, 128, 4, "f16", 0.0),
    "long": ([20000], [1], 10, 2, 128, 5, "bf16", 0.0),
    "capped_long": ([9001, 3], [1, 1], 4, 4, 64, 1, "f16", 5.0),
    "two_tokens": ([30, 0, 129], [2, 3, 2], 4, 4, 128, 1, "f16", 0.0),
    "few_tokens_group": ([30, 0, 129], [4, 7, 1], 16, 4, 128, 4, "bf16", 0.0),
    "chunk": ([0], [200], 2, 2, 128, 1, "f16", 0.0),
    "chunk_edges": ([0, 0, 0, 0, 128, 127, 1], [127, 128, 129, 17, 128, 2, 256], 2, 2, 64, 1, "bf16", 0.0),
    "chunk_group5": ([300, 0, 7], [70, 26, 25], 10, 2, 128, 5, "f16", 0.0),
    "chunk_group8": ([513], [150], 16, 2, 64, 16, "bf16", 0.0),
    "chunk_group7_d80": ([63, 5], [41, 130], 7, 1, 80, 3, "f16", 0.0),
    "chunk_capped": ([100], [140], 4, 2, 128, 2, "bf16", 12.0),
    "chunk_d96": ([33, 0], [200, 1], 3, 3, 96, 1, "f16", 0.0),
    "chunk_d112": ([200], [150], 4, 2, 112, 2, "bf16", 0.0),
    "chunk_group32": ([70, 0], [3, 40], 32, 1, 64, 8, "f16", 0.0),
    "chunk_group33": ([70, 0], [3, 10], 33, 1, 64, 8, "f16", 0.0),
    "chunk_many_short": ([0] * 40, [9 + i % 23 for i in range(40)], 8, 8, 64, 2, "f16", 0.0),
    "decode_group12": ([1000, 3, 128], [1] * 3, 24, 2, 128, 4, "bf16", 0.0),
    "chunk_d256": ([33, 0], [40, 20], 2, 1, 256, 2, "f16", 0.0),
    "chunk_d16": ([5], [300], 4, 4, 16, 4, "bf16", 0.0),
    "mixed": ([9, 600, 0, 77, 0, 300], [1, 1, 90, 1, 400, 33], 8, 4, 128, 2, "bf16", 0.0),
}


@pytest.mark.parametrize("name", ATTEND)
def test_attend_matches_oracle(S, name):
    ctx, new, hq, hkv, d, P, dtype, cap = ATTEND[name]
    s = Setup(S, ctx, new, hq, hkv, d, P, dtype, T=sum(new) + 5)
    _, q, out = _fill_and_attend(S, s, softcap=cap)
    _check_attend(s, q, out, softcap=cap)
    s.close()


def test_attend_layers_and_scale(S):
    s = Setup(S, [50, 3, 0], [1, 20, 64], 4, 2, 64, 4, "f16", layers=3, seed=5)
    _, q, out = _fill_and_attend(S, s, scale=0.3, layer=2)
    _check_attend(s, q, out, scale=0.3, layer=2)
    s.close()


@pytest.mark.parametrize("group", [31, 9])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_bits_do_not_depend_on_earlier_calls(S, group, dtype):
    """Groups that leave rows of a 128-row tile without a query: what an earlier
    call left in their place does not reach the other rows, not even through
    the moment at which their sums are rescaled."""
    # several key tiles in every run; the other call fills all 128 rows
    s = Setup(S, [9000, 7100, 7700], [13, 8, 40], 4 * group, 4, 128, 4, dtype, seed=16)
    s2 = Setup(S, [9000, 7100, 7700], [12, 8, 40], 4 * 32, 4, 128, 4, dtype, seed=17)
    b2, q2, out2 = _fill_and_attend(S, s2)
    b, q, out = _fill_and_attend(S, s)
    for scale in (0.01, 1.0, 100.0):
        s2.kv.attend(b2, 0, (q2 * scale).contiguous(), out2[:, : 4 * 32 * 128])
        again = torch.empty(s.T, 4 * group * 128, dtype=TDT[dtype], device="cuda")
        s.kv.attend(b, 0, q, again)
        assert torch.equal(again.view(torch.int16), out[:, : 4 * group * 128].contiguous().view(torch.int16)), scale
    s.close()
    s2.close()


@pytest.mark.parametrize("new", [1, 64])
def test_attend_peaked_and_equal_scores(S, new):
    """One key far above the rest, and keys that are all the same: the softmax
    at its two ends; scores as large as fp16 products make them."""
    s = Setup(S, [130], [new], 2, 2, 128, 1, "f16", seed=9)
    b = s.plan()
    s.oracle_plan()
    cache = s.cache_rows()
    n = 130 + new
    k = torch.zeros(n, 2, 128, device="cuda")
    k[17, 0], k[:, 1] = 8.0, 1.0
    v = s.randn(n, 256)
    cache[s.slot_rows(0, 0, 0)] = k.view(n, 256).to(torch.float16)
    cache[s.slot_rows(0, 0, 1)] = v
    q = torch.full((new, 256), 8.0, dtype=torch.float16, device="cuda")
    out = torch.full((new, 264), 3.0, dtype=torch.float16, device="cuda")
    s.kv.attend(b, 0, q, out[:, :256])
    torch.cuda.synchronize()
    assert torch.equal(out[:, :128], v[17, :128].expand(new, 128))     # the peak's value, exactly
    _check_attend(s, q, out)
    s.close()


def test_attend_offsets_past_32_bits(S):
    """Rows whose element offsets in the pool are beyond 2^32."""
    s = Setup(S, [40, 200], [1, 70], 8, 8, 128, 64, "f16", first_page=(1 << 32) // (64 * 1024) + 5, seed=3)
    assert s.num_pages * s.H > 1 << 32
    _, q, out = _fill_and_attend(S, s)
    _check_attend(s, q, out)
    s.close()


def test_rows_that_share_a_prefix(S):
    """A row that starts with another row's entries (written by the caller)
    attends over the shared tokens; its own go to its own pages."""
    P, hkv, d, shared = 4, 2, 64, 24
    s = Setup(S, [shared, shared], [1, 9], 4, hkv, d, P, "f16", spare_rows=1)
    n = shared // P
    s.table[:, :, s.rows[1], :n] = s.table[:, :, s.rows[0], :n]
    s.kv.table.copy_(torch.from_numpy(s.table))
    _, q, out = _fill_and_attend(S, s)
    assert (s.table[:, :, s.rows[1], :n] == s.table[:, :, s.rows[0], :n]).all()
    _check_attend(s, q, out)
    s.close()


def test_timing_names_the_kernels(S):
    s = Setup(S, [30, 0], [1, 40], 4, 4, 64, 1, "f16")
    S.slora_timing_enable(s.pool.handle, True)
    _fill_and_attend(S, s)
    t = S.slora_timing_read(s.pool.handle)
    assert t["kv_plan"][1] == 1 and t["kv_attend"][1] == 1 and t["kv_append"][1] == 0 and t["kv_attend"][0] > 0
    s.close()


def test_one_request_not_finite_leaves_the_others(S):
    s = Setup(S, [50, 60, 10], [1, 40, 30], 4, 2, 128, 4, "f16", seed=4)
    b, q, out = _fill_and_attend(S, s)
    good = out.clone()
    s.cache_rows()[s.slot_rows(1, 0, 1)[5]] = float("inf")
    s.cache_rows()[s.slot_rows(1, 0, 0)[9]] = float("nan")
    s.kv.attend(b, 0, q, out[:, : s.hq * s.d])
    torch.cuda.synchronize()
    assert torch.equal(out[:1], good[:1]) and torch.equal(out[41:], good[41:])
    s.close()


def test_attend_is_repeatable(S):
    """The same call twice gives the same bits (splits are joined in a fixed order)."""
    s = Setup(S, [3000, 5, 900, 0], [1, 1, 1, 500], 8, 2, 128, 4, "bf16", seed=6)
    b, q, out = _fill_and_attend(S, s)
    first = out.clone()
    for _ in range(5):
        s.kv.attend(b, 0, q, out[:, : s.hq * s.d])
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    s.close()


def test_step_in_a_cuda_graph(S):
    """plan + append + attend captured once and replayed for steps of other
    lengths, rows and pages: the same bits as the calls made one by one."""
    hq, hkv, d, P, T = 8, 2, 64, 4, 40
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        pool = S.Pool(400, hkv * d * P, "f16", [(8, 8)], 1, 1, T, device=torch.device("cuda", 0), compute_stream=stream)
        kv = S.KVCache(pool, 1, hq, hkv, d, 6, 40)
        kv.set_rotary(d, [1.0 / (i + 1) for i in range(d // 2)])
        pool.buffer.zero_()
        i32 = dict(dtype=torch.int32, device="cuda")
        ctx, new, rows = torch.zeros(3, **i32), torch.zeros(3, **i32), torch.arange(3, **i32)
        pages = torch.zeros(60, **i32)
        qkv = torch.zeros(T, (hq + 2 * hkv) * d, dtype=torch.float16, device="cuda")
        q_out, out = (torch.zeros(T, hq * d, dtype=torch.float16, device="cuda") for _ in range(2))
        w = [hq * d, hkv * d, hkv * d]

        def step():
            b = kv.plan(ctx, new, pages, T, 30, rows=rows)
            q, k, v = qkv.split(w, 1)
            kv.append(b, 0, q, k, v, q_out=q_out)
            kv.attend(b, 0, q_out, out)

        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        held, nxt = np.zeros(3, np.int64), 0
        for lens in ([5, 30, 1], [1, 1, 1], [1, 0, 12], [30, 1, 1]):
            lens = np.array(lens)
            opened = int(sum(-(-(h + n) // P) - -(-h // P) for h, n in zip(held, lens)))
            ctx.copy_(torch.from_numpy(held.astype(np.int32)))
            new.copy_(torch.from_numpy(lens.astype(np.int32)))
            pages[: 2 * opened].copy_(torch.arange(nxt, nxt + 2 * opened, dtype=torch.int32))
            nxt += 2 * opened
            qkv.normal_()
            kept = pool.buffer.clone(), kv.table.clone()
            graph.replay()
            got = out.clone(), pool.buffer.clone()
            pool.buffer.copy_(kept[0])
            kv.table.copy_(kept[1])
            out.zero_()
            step()
            n = int(lens.sum())
            stream.synchronize()
            assert torch.equal(out[:n], got[0][:n]) and torch.equal(pool.buffer, got[1])
            held += lens
        assert pool.status() == S.OK
    stream.synchronize()
    kv.close()
    pool.close()


def test_refusals(S):
    def err(f, *a, code=None, **kw):
        with pytest.raises(S.SloraError) as e:
            f(*a, **kw)
        assert e.value.code == (S.ERR_INVALID if code is None else code)

    pool = S.Pool(20, 1024, "f16", [(8, 8)], 1, 1, 8, device=torch.device("cuda", 0))
    good = {"layers": 1, "heads_q": 4, "heads_kv": 2, "head_dim": 64, "max_requests": 4, "max_blocks": 4}
    for bad in (dict(layers=0), dict(heads_kv=0), dict(heads_q=3), dict(heads_q=1), dict(head_dim=24),
                dict(head_dim=272), dict(head_dim=0), dict(heads_q=6, heads_kv=6, head_dim=80), dict(max_requests=0),
                dict(max_requests=4097), dict(max_blocks=0), dict(max_blocks=1 << 29)):
        err(S.slora_kv_create, pool.handle, *(good | bad).values(), pool.buffer.data_ptr(), pool.buffer.data_ptr())
        err(S.slora_kv_array_ints, pool.handle, *(good | bad).values())
    some = pool.buffer.data_ptr()
    err(S.slora_kv_create, pool.handle, *good.values(), 0, some)
    err(S.slora_kv_create, pool.handle, *good.values(), some, 0)
    err(S.slora_kv_create, 0, *good.values(), some, some)
    kv = S.KVCache(pool, **good)
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new = torch.zeros(2, **i32), torch.ones(2, **i32)
    pages = torch.arange(4, **i32)
    err(kv.plan, ctx, new, pages, 9, 1)                  # more tokens than the pool's max_tokens
    err(kv.plan, ctx, new, pages, -1, 1)
    err(kv.plan, ctx, new, pages, 2, -1)
    err(kv.plan, ctx, new, pages[:3], 2, 1)              # not whole blocks
    err(kv.plan, torch.zeros(5, **i32), torch.zeros(5, **i32), pages, 2, 1)   # more requests than rows
    with pytest.raises(ValueError):
        kv.plan(ctx.long(), new, pages, 2, 1)
    with pytest.raises(ValueError):
        kv.plan(ctx, new[:1], pages, 2, 1)
    f = [1.0] * 32
    err(kv.set_rotary, 24, f)
    err(kv.set_rotary, 80, f + f)
    err(kv.set_rotary, 64, [float("inf")] * 32)
    err(kv.set_rotary, 64, f, mscale=float("nan"))
    err(S.slora_kv_set_rotary, kv.handle, 64, 2, f)
    b0 = kv.plan(ctx, new, pages, 2, 1)
    b = kv.plan(ctx, new, pages, 2, 1)
    q, k, v, out = z(2, 256), z(2, 128), z(2, 128), z(2, 256)
    err(kv.attend, b0, 0, q, out)                        # stale
    err(kv.append, b0, 0, q, k, v)
    err(kv.attend, b, 1, q, out)                         # no such layer
    err(kv.append, b, -1, q, k, v)
    err(kv.attend, b, 0, q, out, softcap=-1.0)
    err(kv.attend, b, 0, q, out, scale=float("nan"))
    err(kv.attend, b, 0, q, out, scale=0.0)
    err(kv.attend, b, 0, q, out, scale=-1.0)
    err(kv.attend, b, 0, z(2, 260)[:, 1:257], out)       # not 16-byte aligned
    err(kv.attend, b, 0, z(2, 257)[:, :256], out)        # row stride not a multiple of 8
    err(kv.append, b, 0, q, k, v, q_weight=z(64))        # weights go together
    err(kv.append, b, 0, q, k, v, q_weight=z(64), k_weight=z(64), eps=-1.0)
    with pytest.raises(ValueError):
        kv.attend(b, 0, q.bfloat16(), out)
    with pytest.raises(ValueError):
        kv.attend(b, 0, q[:1], out)
    with pytest.raises(ValueError):
        kv.append(b, 0, q, k, v, q_weight=z(32), k_weight=z(64))
    kv.append(b, 0, q, k, v)
    kv.attend(b, 0, q, out)
    assert pool.status() == S.OK
    kv.close()
    pool.close()
