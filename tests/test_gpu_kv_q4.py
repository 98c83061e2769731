"""Key-value caches held in 4 bits on the GPU against the fp64 oracle:
slora_kv_append, slora_kv_attend and slora_kv_read on a slora_kv_q4_create handle.

Tolerances.  u is the largest relative error of one rounding to the storage
type (fp16 2^-11, bf16 2^-8).
 - append: the bytes of the oracle, all of them (codes are chosen as in exact
   arithmetic); queries as in a 16-bit cache, u |y| + 2^-18 of the largest.
 - read: the stored numbers, exactly.
 - attend: one rounding of the result, u |o|; scores of at most 256 fp32
   products and the softmax leave 2^-12 of the largest |v| of the request's
   head; requests with more than 8 rows (new tokens times query heads a key
   head) may round the weights to the storage type, u of it.
"""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from oracle import kv_q4 as oq4

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
    """A pool of pages whose bytes are all 0xff (every M a NaN) and a 4-bit cache
    with the requests' context blocks in its table."""

    def __init__(self, S, ctx, new, hq, hkv, d, page_elems, dtype, layers=1, seed=0, spare_rows=2, T=None,
                 first_page=0, num_pages=None):
        self.S = S
        rng = np.random.default_rng(seed)
        self.rng, self.g = rng, torch.Generator(device="cuda").manual_seed(seed)
        self.rb = oq4.row_bytes(hkv, d)
        P = 2 * page_elems // self.rb
        self.ctx, self.new, self.P, self.L, self.d, self.hq, self.hkv = ctx, new, P, layers, d, hq, hkv
        self.dtype, self.page_elems = dtype, page_elems
        R = len(ctx)
        self.T = sum(new) if T is None else T
        blocks = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        n_blocks = sum(blocks)
        self.num_pages = num_pages or first_page + n_blocks * 2 * layers + 3
        self.pages = (rng.permutation(n_blocks * 2 * layers + 3)[: n_blocks * 2 * layers] + first_page).reshape(
            n_blocks, layers, 2)
        self.pool = S.Pool(self.num_pages, page_elems, dtype, [(8, 8)], 1, 1, max(self.T, 1),
                           device=torch.device("cuda", 0))
        self.pool.buffer[first_page:].view(torch.int16).fill_(-1)
        max_rows = R + spare_rows
        self.rows = rng.permutation(max_rows)[:R].astype(np.int32)
        self.max_blocks = max(blocks + [1])
        self.kv = S.KVCache(self.pool, layers, hq, hkv, d, max(1, max_rows), self.max_blocks, bits=4)
        assert self.kv.tokens_per_page == P
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

    def row_view(self):
        """The pool as token rows: [page, token of the page, byte]."""
        return self.pool.buffer.view(torch.uint8).as_strided((self.num_pages, self.P, self.rb),
                                                             (2 * self.page_elems, self.rb, 1))

    def at(self, r, layer, j, n=None):
        """(pages, tokens of the page) of the n tokens request r holds after the step."""
        p = np.arange(self.ctx[r] + self.new[r] if n is None else n)
        page = self.table[layer, j, self.rows[r], p // self.P].astype(np.int64)
        return torch.from_numpy(page).cuda(), torch.from_numpy(p % self.P).cuda()

    def fill(self, layer=0, spread=1.0):
        """Stores random tokens for every request: the numbers they stand for, [r] -> (keys, values)."""
        view, out = self.row_view(), []
        for r in range(len(self.ctx)):
            n, got = self.ctx[r] + self.new[r], []
            for j in (0, 1):
                ng = oq4.groups(self.d)
                k = self.rng.integers(-7, 9, (n, self.hkv, 32 * ng))
                M = np.vectorize(lambda m: oq4.scale(m, self.dtype), otypes=[np.float64])(
                    self.rng.standard_normal((n, self.hkv, ng)) * spread)
                if n:
                    rows = oq4.pack(k, M, self.dtype, j == 1)
                    assert np.array_equal(oq4.unpack(rows, self.hkv, self.d, self.dtype, j == 1), oq4.values(k, M, self.d))
                    view[self.at(r, layer, j)] = torch.from_numpy(rows).cuda()
                got.append(oq4.values(k, M, self.d))
            out.append(got)
        return out

    def close(self):
        self.kv.close()
        self.pool.close()


ROT = {   # rot_dim (0: all), interleaved, norm, mscale, factor
    "half": (0, False, False, 1.0, 1.0),
    "half_norm": (0, False, True, 1.0, 1.0),
    "interleaved": (0, True, False, 1.0, 1.0),
    "interleaved_norm_scaled": (0, True, True, 1.25, 8.0),
    "part": (32, False, True, 1.0, 1.0),
    "part_interleaved": (16, True, False, 0.5, 1.0),
    "part_half": (16, False, False, 1.0, 1.0),
    "norm_only": (-1, False, True, 1.0, 1.0),
    "copy": (-1, False, False, 1.0, 1.0),
}


@pytest.mark.parametrize("rot", ROT)
@pytest.mark.parametrize("dtype,hq,hkv,d,H", [("f16", 4, 4, 64, 256), ("bf16", 10, 2, 128, 1280), ("f16", 3, 1, 80, 88),
                                              ("bf16", 2, 1, 256, 768), ("f16", 7, 7, 16, 72), ("bf16", 4, 2, 96, 760),
                                              ("f16", 6, 3, 128, 128 * 3)])
def test_append_stores_the_oracles_bytes(S, rot, dtype, hq, hkv, d, H):
    rot_dim, inter, norm, mscale, factor = ROT[rot]
    rot_dim = d if rot_dim == 0 else max(0, min(rot_dim, d))
    ctx, new, layers = [0, 1, 131071, 40], [9, 1, 2, 0], 2
    s = Setup(S, ctx, new, hq, hkv, d, H, dtype, layers=layers, T=14)
    freq = [10000.0 ** (-2 * i / max(rot_dim, 1)) / factor for i in range(rot_dim // 2)]
    s.kv.set_rotary(rot_dim, freq, interleaved=inter, mscale=mscale)
    b = s.plan()
    want = s.oracle_plan()
    T, layer = s.T, 1
    qkv = s.randn(T, (hq + 2 * hkv) * d + 8)
    q, k, v = qkv[:, : hq * d], qkv[:, hq * d: (hq + hkv) * d], qkv[:, (hq + hkv) * d: (hq + 2 * hkv) * d]
    qw, kw = (s.randn(d, scale=0.3) + 1, s.randn(d, scale=0.3) + 1) if norm else (None, None)
    q_out = torch.full((T, hq * d + 16), 7.0, dtype=TDT[dtype], device="cuda")
    before = s.pool.buffer.view(torch.uint8).clone()
    s.kv.append(b, layer, q, k, v, q_out=q_out[:, : hq * d], q_weight=qw, k_weight=kw, eps=1e-5)
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    n_tok, ng = sum(new), oq4.groups(d)
    expect = before.clone().cpu().numpy().reshape(s.num_pages, -1)
    for t in range(n_tok):
        pos = int(want["tok_pos"][t])
        y = okv.norm_rotate(f64(q[t]).reshape(hq, d), f64(qw) if norm else None, 1e-5, pos, freq, rot_dim, inter, mscale)
        err = np.abs(f64(q_out[t, : hq * d]).reshape(hq, d) - y)
        assert (err <= U[dtype] * np.abs(y) + 2.0 ** -18 * max(1.0, np.abs(y).max())).all(), (t, err.max())
        kk = okv.norm_rotate(f64(k[t]).reshape(hkv, d), f64(kw) if norm else None, 1e-5, pos, freq, rot_dim, inter, mscale)
        for j, x in ((0, kk), (1, f64(v[t]).reshape(hkv, d))):
            slot = int(want["slots"][layer, j, t])
            row = oq4.pack(*(z[None] for z in oq4.quantise(x, dtype)), dtype, j == 1)[0]
            at = slot % s.P * s.rb
            expect[slot // s.P, at: at + 18 * ng * hkv] = row[: 18 * ng * hkv]
    got = s.pool.buffer.view(torch.uint8).cpu().numpy().reshape(s.num_pages, -1)
    assert np.array_equal(got, expect)             # the tokens' rows, and nothing else
    assert (q_out[n_tok:] == 7).all() and (q_out[:, hq * d:] == 7).all()
    # in place gives the same bits
    qi = qkv.clone()
    s.kv.append(b, layer, qi[:, : hq * d], k, v, q_weight=qw, k_weight=kw, eps=1e-5)
    assert torch.equal(qi[:n_tok, : hq * d], q_out[:n_tok, : hq * d])
    assert np.array_equal(s.pool.buffer.view(torch.uint8).cpu().numpy().reshape(s.num_pages, -1), expect)
    s.close()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_codes_at_their_borders(S, dtype):
    """Values on, just below and just above every border between two codes, for every
    M of five significant bits and both signs; groups of zeros, of both signs at the
    same magnitude, of the smallest numbers and of the largest."""
    d, u = 128, U[dtype]
    rows = []
    for n in range(16, 32):
        for sign in (1.0, -1.0):
            M = sign * n / 16.0
            border = M * (2 * np.arange(-8, 8) + 1) / 16
            lo = np.concatenate([[M], border[1:], border[1:] * (1 - 2 * u)])
            hi = np.concatenate([[M], border[1:], border[1:] * (1 + 2 * u)])
            rows.append(np.concatenate([np.resize(lo, 32), np.resize(hi, 32), np.resize(lo, 32) * 2.0 ** -9,
                                        np.resize(hi, 32) * 2.0 ** 9]))
    tiny, top = (2.0 ** -24, 65504.0) if dtype == "f16" else (2.0 ** -133, 3.3895313892515355e38)
    rng = np.random.default_rng(3)
    even = np.linspace(-1, 1, 32)
    rows += [np.zeros(d), np.tile(np.where(np.arange(32) % 2, 1.0, -1.0), 4), -np.tile(even, 4)[::-1],
             rng.integers(-40, 41, d) * tiny, np.full(d, tiny), rng.uniform(-1, 1, d) * top, np.full(d, -top),
             np.tile(even, 4) * top, np.where(np.arange(d) % 7, 0.0, 1.0), rng.integers(-3, 4, d) * 2.0 ** -17]
    x = torch.from_numpy(np.array(rows)).to(TDT[dtype]).cuda()
    n = x.shape[0]
    s = Setup(S, [0], [n], 1, 1, d, 400, dtype)
    b = s.plan()
    s.oracle_plan()
    q = s.randn(n, d)
    s.kv.append(b, 0, q, x, x)                     # no norm, no rotation: keys too are as they come
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    for j in (0, 1):
        got = s.row_view()[s.at(0, 0, j)].cpu().numpy()
        for t in range(n):
            k, M = oq4.quantise(f64(x[t]).reshape(1, d), dtype)
            assert np.array_equal(got[t, :72], oq4.pack(k[None], M[None], dtype, j == 1)[0, :72]), (j, t, k, M)
            held = f64(x[t]).reshape(1, d)
            assert (np.abs(oq4.values(k, M, d) - held) <= np.abs(np.repeat(M, 32, -1)) / 8 + 2.0 ** -30).all() or t >= 32
    s.close()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rotate", [False, True])
def test_groups_that_are_not_finite(S, dtype, rotate):
    """A NaN or an infinity makes its group of 32 NaN, and no other (a rotated pair: both
    elements' groups)."""
    d, T = 128, 4
    s = Setup(S, [3], [T], 2, 2, d, 600, dtype)
    if rotate:
        s.kv.set_rotary(64, [10000.0 ** (-2 * i / 64) for i in range(32)])
    b = s.plan()
    s.oracle_plan()
    q, k, v = s.randn(T, 2 * d), s.randn(T, 2 * d), s.randn(T, 2 * d)
    k[0, 5], k[1, d + 70], v[2, 127], v[3, d] = float("nan"), float("inf"), float("-inf"), float("nan")
    s.kv.append(b, 0, q, k, v)
    out_k, out_v = torch.zeros(T, 2 * d, dtype=TDT[dtype], device="cuda"), torch.zeros(T, 2 * d, dtype=TDT[dtype], device="cuda")
    s.kv.read(0, s.dev([s.rows[0]] * T), s.dev(range(3, 3 + T)), out_k, out_v)
    bad_k, bad_v = torch.zeros(T, 8, dtype=torch.bool), torch.zeros(T, 8, dtype=torch.bool)
    bad_k[0, 0] = bad_k[1, 6] = bad_v[2, 3] = bad_v[3, 4] = True
    if rotate:
        bad_k[0, 1] = True                         # the pair's other half
    assert torch.equal(out_k.isnan().view(T, 8, 32).all(-1).cpu(), bad_k) and torch.equal(out_k.isnan().view(T, 8, 32).any(-1).cpu(), bad_k)
    assert torch.equal(out_v.isnan().view(T, 8, 32).all(-1).cpu(), bad_v) and torch.equal(out_v.isnan().view(T, 8, 32).any(-1).cpu(), bad_v)
    assert s.pool.status() == S.OK
    s.close()


READ = {   # hq, hkv, d, page_elems, dtype
    "mha": (4, 4, 128, 512, "f16"),
    "gqa": (10, 2, 128, 1288, "bf16"),
    "d80": (3, 1, 80, 88, "f16"),
    "d256": (2, 1, 256, 776, "bf16"),
    "d16": (7, 7, 16, 72, "f16"),
    "d96": (4, 2, 96, 768, "bf16"),
}


@pytest.mark.parametrize("name", READ)
def test_read_gives_the_stored_numbers(S, name):
    hq, hkv, d, H, dtype = READ[name]
    s = Setup(S, [70, 1, 0, 33], [0, 0, 0, 2], hq, hkv, d, H, dtype, layers=2)
    b = s.plan()
    s.oracle_plan()
    held = s.fill(layer=1)
    pick = [(r, p) for r in (0, 1, 3) for p in range(s.ctx[r] + s.new[r])]
    s.rng.shuffle(pick)
    pick += pick[:5] + [(0, -1), (3, -7)]          # the same token twice, and rows without one
    rows, pos = s.dev([s.rows[r] for r, _ in pick]), s.dev([p for _, p in pick])
    n = len(pick)
    k = torch.full((n, hkv * d + 16), 5.0, dtype=TDT[dtype], device="cuda")
    v = torch.full((n, hkv * d + 24), 5.0, dtype=TDT[dtype], device="cuda")
    s.kv.read(1, rows, pos, k[:, 8: 8 + hkv * d], v[:, : hkv * d])
    torch.cuda.synchronize()
    assert s.pool.status() == S.OK
    for i, (r, p) in enumerate(pick):
        for j, got in ((0, k[i, 8: 8 + hkv * d]), (1, v[i, : hkv * d])):
            if p < 0:
                assert (got == 5).all()
            else:
                assert np.array_equal(f64(got).reshape(hkv, d), held[r][j][p]), (i, r, p, j)
    assert (k[:, :8] == 5).all() and (k[:, 8 + hkv * d:] == 5).all() and (v[:, hkv * d:] == 5).all()
    only = torch.zeros(n, hkv * d, dtype=TDT[dtype], device="cuda")
    s.kv.read(1, rows, pos, v=only)
    assert torch.equal(only[:-2], v[:-2, : hkv * d])
    s.kv.read(1, rows, pos, k=only)
    assert torch.equal(only[:-2], k[:-2, 8: 8 + hkv * d])
    s.kv.read(1, rows[:0], pos[:0], only[:0], only[:0].clone())
    s.close()


def test_read_of_a_16_bit_cache_gives_its_bits(S):
    hkv, d, P, dtype = 3, 48, 5, "bf16"
    pool = S.Pool(20, hkv * d * P, dtype, [(8, 8)], 1, 1, 8, device=torch.device("cuda", 0))
    kv = S.KVCache(pool, 1, hkv, hkv, d, 4, 3)
    pool.buffer.copy_(torch.randn(20, hkv * d * P, device="cuda"))
    table = torch.randperm(20)[:2 * 3].view(2, 3).to(torch.int32)
    kv.table[0, :, 2] = table.cuda()
    pos = torch.arange(13, dtype=torch.int32, device="cuda")
    rows = torch.full_like(pos, 2)
    k, v = (torch.empty(13, hkv * d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kv.read(0, rows, pos, k, v)
    assert pool.status() == S.OK
    for j, got in ((0, k), (1, v)):
        for p in range(13):
            row = pool.buffer[int(table[j, p // P])].view(P, -1)[p % P]
            assert torch.equal(got[p].view(torch.int16), row.view(torch.int16))
    kv.close()
    pool.close()


def test_read_reports_what_it_cannot_find(S):
    s = Setup(S, [20, 9], [0, 0], 2, 2, 64, 304, "f16")
    s.fill()
    width = s.max_blocks * s.P
    for name, row, p in (("row outside", len(s.rows) + 2, 0), ("row below", -1, 0), ("position past the table", 0, width),
                         ("far position", 0, 2 ** 31 - 1), ("no such page", int(s.rows[1]), 20)):
        out = torch.full((3, 128), 5.0, dtype=torch.float16, device="cuda")
        v = out.clone()
        s.kv.read(0, s.dev([s.rows[0], row, s.rows[0]]), s.dev([3, p, 4]), out, v)
        assert s.pool.status() == S.ERR_INVALID, name
        assert (out[1] == 5).all() and (v[1] == 5).all() and not (out[[0, 2]] == 5).all(), name
    s.kv.table[0, 1, int(s.rows[0]), 0] = s.num_pages       # V's entry alone
    out = torch.full((1, 128), 5.0, dtype=torch.float16, device="cuda")
    v = out.clone()
    s.kv.read(0, s.dev([s.rows[0]]), s.dev([0]), out, v)
    assert s.pool.status() == S.ERR_INVALID and (v == 5).all() and not (out == 5).all()
    s.close()


def _attend(s, held, softcap=0.0, scale=None, layer=0, requests=None):
    b = s.plan()
    hq, hkv, d, T = s.hq, s.hkv, s.d, s.T
    q = s.randn(T, hq * d + 24, scale=2.0)[:, 8: 8 + hq * d]
    out = torch.full((T, hq * d + 8), 3.0, dtype=TDT[s.dtype], device="cuda")
    s.kv.attend(b, layer, q, out[:, : hq * d], scale=scale, softcap=softcap)
    torch.cuda.synchronize()
    assert s.pool.status() == S_OK
    _check(s, held, q, out, softcap, scale, requests)
    return b, q, out


S_OK = 0


def _check(s, held, q, out, softcap=0.0, scale=None, requests=None):
    hq, hkv, d = s.hq, s.hkv, s.d
    scale = d ** -0.5 if scale is None else scale
    decode = max(s.new + [0]) * (hq // hkv) <= 8
    t0 = 0
    for r, (c, n) in enumerate(zip(s.ctx, s.new)):
        if n and (requests is None or r in requests):
            keys, vals = held[r]
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
    # ctx, new, hq, hkv, d, page_elems, dtype, softcap
    "one_token": ([0], [1], 4, 4, 64, 256, "f16", 0.0),
    "one_key_head": ([777], [1], 8, 1, 128, 512, "bf16", 0.0),
    "decode": ([0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 200, 1000], [1] * 12, 8, 8, 128, 1024, "f16", 0.0),
    "decode_bf16": ([0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 200, 1000], [1] * 12, 8, 8, 128, 1024, "bf16", 0.0),
    "decode_heads32": ([0, 3, 130, 511, 900], [1] * 5, 32, 32, 128, 4096, "f16", 0.0),
    "decode_group2": ([0, 3, 130, 511, 90], [1] * 5, 8, 4, 128, 520, "f16", 0.0),
    "decode_group4": ([0, 3, 130, 511, 90], [1] * 5, 16, 4, 128, 520, "bf16", 0.0),
    "decode_group5": ([0, 3, 130, 511, 900], [1] * 5, 20, 4, 128, 2560, "bf16", 0.0),
    "decode_group16": ([40, 333], [1, 1], 32, 2, 64, 1024, "f16", 0.0),
    "decode_group24": ([40, 333], [1, 1], 24, 1, 64, 512, "f16", 30.0),
    "decode_d64": ([12, 90, 257], [1] * 3, 12, 3, 64, 400, "bf16", 0.0),
    "decode_d80": ([12, 90, 257], [1] * 3, 6, 3, 80, 480, "f16", 0.0),
    "decode_d96_mha": ([12, 90, 257], [1] * 3, 3, 3, 96, 480, "f16", 0.0),
    "decode_d96_group4": ([12, 90, 257], [1] * 3, 12, 3, 96, 480, "bf16", 0.0),
    "decode_d80_mha5": ([12, 90, 257, 700], [1] * 4, 5, 5, 80, 480, "f16", 0.0),
    "decode_d80_two": ([12, 90, 257], [2, 1, 2], 3, 3, 80, 480, "bf16", 30.0),
    "mixed_d96": ([9, 600, 33, 77], [1, 8, 90, 5], 3, 3, 96, 480, "f16", 0.0),
    "decode_d48": ([12, 90, 257], [1] * 3, 4, 4, 48, 480, "f16", 0.0),
    "decode_d32": ([12, 90, 257], [1, 3, 2], 8, 2, 32, 480, "bf16", 0.0),
    "decode_d160": ([12, 90, 257], [1] * 3, 8, 4, 160, 800, "f16", 30.0),
    "decode_seven_heads": ([12, 90, 2570], [1] * 3, 7, 7, 256, 1536, "f16", 0.0),
    "decode_five_heads": ([12, 900, 2570], [1] * 3, 10, 5, 192, 1280, "bf16", 0.0),
    "decode_eleven_heads": ([12, 900, 2570], [1, 2, 1], 22, 11, 64, 1280, "f16", 20.0),
    "decode_thirteen_heads": ([1200, 0, 2570], [1] * 3, 13, 13, 128, 2048, "bf16", 0.0),
    "chunk_over_long": ([20000, 300], [40, 9], 8, 2, 128, 1280, "f16", 0.0),
    "chunk_over_long_d96": ([9000, 1], [60, 200], 6, 3, 96, 1280, "bf16", 0.0),
    "decode_d176": ([12, 90, 257], [1] * 3, 4, 2, 176, 800, "bf16", 0.0),
    "decode_d224": ([12, 90, 257], [1] * 3, 3, 3, 224, 800, "f16", 0.0),
    "decode_d256": ([12, 90, 257], [1] * 3, 4, 2, 256, 1536, "bf16", 20.0),
    "decode_d256_mha": ([12, 90, 257], [1] * 3, 2, 2, 256, 1536, "f16", 0.0),
    "decode_d240": ([12, 90, 257], [1] * 3, 8, 1, 240, 700 // 8 * 8, "f16", 0.0),
    "decode_d16": ([100, 7], [1, 1], 3, 3, 16, 336, "f16", 0.0),
    "decode_heads20": ([100, 7, 64], [1] * 3, 20, 20, 64, 1280, "bf16", 0.0),
    "decode_heads5": ([100, 7, 640], [1] * 3, 5, 5, 128, 640, "bf16", 0.0),
    "some_none": ([5, 80, 0, 0, 31], [1, 0, 0, 1, 1], 8, 2, 128, 1024, "f16", 0.0),
    "long": ([20000], [1], 10, 2, 128, 1280, "bf16", 0.0),
    "capped_long": ([9001, 3], [1, 1], 4, 4, 64, 256, "f16", 5.0),
    "two_tokens": ([30, 0, 129], [2, 3, 2], 4, 4, 128, 512, "f16", 0.0),
    "two_tokens_each": ([30, 1, 129], [2, 2, 1], 4, 4, 128, 512, "bf16", 0.0),
    "few_tokens_group": ([30, 0, 129], [4, 7, 1], 16, 4, 128, 2048, "bf16", 0.0),
    "chunk": ([0], [200], 2, 2, 128, 256, "f16", 0.0),
    "chunk_edges": ([0, 0, 0, 0, 128, 127, 1], [127, 128, 129, 17, 128, 2, 256], 2, 2, 64, 128, "bf16", 0.0),
    "chunk_group5": ([300, 0, 7], [70, 26, 25], 10, 2, 128, 1280, "f16", 0.0),
    "chunk_group8": ([513], [150], 16, 2, 64, 2048, "bf16", 0.0),
    "chunk_group7_d80": ([63, 5], [41, 130], 7, 1, 80, 240, "f16", 0.0),
    "chunk_capped": ([100], [140], 4, 2, 128, 512, "bf16", 12.0),
    "chunk_capped_far": ([100], [140], 4, 2, 128, 512, "f16", 120.0),
    "chunk_d96": ([33, 0], [200, 1], 3, 3, 96, 288, "f16", 0.0),
    "chunk_d112": ([200], [150], 4, 2, 112, 448, "bf16", 0.0),
    "chunk_group32": ([70, 0], [3, 40], 32, 1, 64, 512, "f16", 0.0),
    "chunk_group33": ([70, 0], [3, 10], 33, 1, 64, 512, "f16", 0.0),
    "chunk_many_short": ([0] * 40, [9 + i % 23 for i in range(40)], 8, 8, 64, 1024, "f16", 0.0),
    "decode_group12": ([1000, 3, 128], [1] * 3, 24, 2, 128, 1024, "bf16", 0.0),
    "chunk_d256": ([33, 0], [40, 20], 2, 1, 256, 512, "f16", 0.0),
    "chunk_d16": ([5], [300], 4, 4, 16, 256, "bf16", 0.0),
    "mixed": ([9, 600, 0, 77, 0, 300], [1, 1, 90, 1, 400, 33], 8, 4, 128, 1024, "bf16", 0.0),
    "mixed_tiles_of_2": ([9, 600, 33, 77, 0, 300], [1, 8, 3, 5, 100, 2], 4, 4, 128, 520, "f16", 0.0),
    "mixed_tiles_of_4": ([9, 600, 33, 77, 0, 300], [2, 1, 2, 1, 50, 2], 12, 3, 128, 520, "bf16", 0.0),
    "mixed_tiles_of_4_d64": ([9, 600, 33, 77, 0, 300], [1, 8, 3, 5, 100, 2], 4, 4, 64, 520, "f16", 30.0),
    "mixed_d256": ([9, 600, 33], [1, 3, 2], 3, 3, 256, 1024, "f16", 0.0),
    "mixed_mha": ([9, 600, 0, 77, 0, 300], [1, 1, 90, 1, 400, 33], 4, 4, 128, 520, "f16", 0.0),
}


@pytest.mark.parametrize("name", ATTEND)
def test_attend_matches_oracle(S, name):
    ctx, new, hq, hkv, d, H, dtype, cap = ATTEND[name]
    s = Setup(S, ctx, new, hq, hkv, d, H, dtype, T=sum(new) + 5)
    s.oracle_plan()
    _attend(s, s.fill(), softcap=cap)
    s.close()


def test_attend_layers_and_scale(S):
    s = Setup(S, [50, 3, 0], [1, 20, 64], 4, 2, 64, 512, "f16", layers=3, seed=5)
    s.oracle_plan()
    _attend(s, s.fill(layer=2), scale=0.3, layer=2)
    s.close()


def test_offsets_past_32_bits(S):
    """Rows whose byte offsets in the pool are beyond 2^33: append, attend and read."""
    H = 64 * 1024
    s = Setup(S, [40, 200], [1, 70], 8, 8, 128, H, "f16", first_page=(1 << 33) // (2 * H) + 5, seed=3)
    s.oracle_plan()
    held = s.fill()
    b, q, out = _attend(s, held)
    x = s.randn(s.T, 8 * 128)
    s.kv.append(b, 0, q, x, x, q_out=torch.empty_like(x))
    k, v = torch.empty_like(x), torch.empty_like(x)
    s.kv.read(0, s.dev([s.rows[0]] + [s.rows[1]] * 70), s.dev([40] + list(range(200, 270))), k, v)
    assert torch.equal(k, v) and s.pool.status() == S.OK
    kq = [oq4.values(*oq4.quantise(f64(x[t]).reshape(8, 128), "f16"), 128) for t in (0, 70)]
    assert np.array_equal(f64(k[[0, 70]]).reshape(2, 8, 128), np.array(kq))
    s.close()


@pytest.mark.parametrize("dtype,hq,hkv,d,H", [("f16", 8, 8, 128, 1024), ("bf16", 10, 2, 64, 640)])
def test_a_request_grown_over_steps(S, dtype, hq, hkv, d, H):
    """Plan, append, attend and read together: two requests grown by prompt chunks and
    single tokens, each step's attention against the oracle over what the cache holds."""
    L, steps = 2, [(40, 7), (1, 1), (19, 1), (1, 30), (1, 1)]
    rb = oq4.row_bytes(hkv, d)
    P = 2 * H // rb
    pool = S.Pool(300, H, dtype, [(8, 8)], 1, 1, 80, device=torch.device("cuda", 0))
    pool.buffer.view(torch.int16).fill_(-1)
    kv = S.KVCache(pool, L, hq, hkv, d, 4, 40, bits=4)
    freq = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    kv.set_rotary(d, freq)
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    ctx, perm, used = np.zeros(2, np.int64), np.random.default_rng(0).permutation(300), 0
    stored = [[[], []], [[], []]]                  # [request][K, V] of layer 1, fp64 after 4 bits
    for new in steps:
        new = np.array(new)
        opened = int(sum(-(-(c + n) // P) - -(-c // P) for c, n in zip(ctx, new)))
        pages = torch.from_numpy(perm[used: used + opened * 2 * L].astype(np.int32)).cuda()
        used += opened * 2 * L
        T = int(new.sum())
        i32 = lambda x: torch.tensor([int(y) for y in x], dtype=torch.int32, device="cuda")
        b = kv.plan(i32(ctx), i32(new), pages, T, int(new.max()), rows=rows)
        for layer in range(L):
            qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda").to(TDT[dtype])
            q, k, v = qkv[:, : hq * d], qkv[:, hq * d: (hq + hkv) * d], qkv[:, (hq + hkv) * d:]
            q_rot, out = torch.empty(T, hq * d, dtype=TDT[dtype], device="cuda"), torch.empty(T, hq * d, dtype=TDT[dtype], device="cuda")
            kv.append(b, layer, q, k, v, q_out=q_rot)
            kv.attend(b, layer, q_rot, out)
        t0 = 0
        for r in range(2):
            for i in range(new[r]):
                kk = okv.norm_rotate(f64(k[t0 + i]).reshape(hkv, d), None, 0.0, int(ctx[r]) + i, freq, d, False, 1.0)
                stored[r][0].append(oq4.values(*oq4.quantise(kk, dtype), d))
                stored[r][1].append(oq4.values(*oq4.quantise(f64(v[t0 + i]).reshape(hkv, d), dtype), d))
            keys, vals = np.array(stored[r][0]), np.array(stored[r][1])
            n = int(ctx[r] + new[r])
            rk, rv = (torch.empty(n, hkv * d, dtype=TDT[dtype], device="cuda") for _ in "kv")
            kv.read(1, torch.full((n,), int(rows[r]), dtype=torch.int32, device="cuda"),
                    torch.arange(n, dtype=torch.int32, device="cuda"), rk, rv)
            assert np.array_equal(f64(rk).reshape(n, hkv, d), keys) and np.array_equal(f64(rv).reshape(n, hkv, d), vals)
            want = okv.attend(f64(q_rot[t0: t0 + new[r]]).reshape(-1, hq, d), keys, vals, int(ctx[r]), d ** -0.5, 0.0)
            err = np.abs(f64(out[t0: t0 + new[r]]).reshape(-1, hq, d) - want)
            assert (err <= U[dtype] * np.abs(want) + (2.0 ** -12 + U[dtype]) * np.abs(vals).max()).all()
            t0 += int(new[r])
        ctx = ctx + new
    assert pool.status() == S.OK
    kv.close()
    pool.close()


def test_normed_keys_of_equal_magnitude_take_the_positive_sign(S):
    """Elements whose products with the norm's weights have the same magnitude and
    different signs: the tie is exact, whatever rounding the norm brings."""
    d, n, dtype = 64, 300, "bf16"
    s = Setup(S, [0], [n], 1, 1, d, 400, dtype)
    b = s.plan()
    s.oracle_plan()
    k = s.randn(n, d).clamp(-2, 2)
    w = torch.full((d,), 1.0, dtype=torch.bfloat16, device="cuda")
    w[3], w[40] = 0.75, 0.75
    k[:, 3], k[:, 17], k[:, 40], k[:, 61] = -4.0, 3.0, 4.0, -3.0      # 0.75 * 4 = 3
    s.kv.append(b, 0, k.clone(), k, k, q_out=torch.empty_like(k), q_weight=w, k_weight=w)
    out = torch.empty_like(k)
    s.kv.read(0, s.dev([s.rows[0]] * n), s.dev(range(n)), out)
    # m is the positive one: it becomes M itself, the negative one at most 7 / 8 of M
    assert (out[:, 17] == -out[:, 3] * 8 / 7).all() and (out[:, 40] == -out[:, 61] * 8 / 7).all() and (out[:, 17] > 0).all()
    assert s.pool.status() == S.OK
    s.close()
