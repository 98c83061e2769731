"""CPU tests of the paged key-value cache: what the host refuses before any
CUDA call, and the fp64 oracle against closed forms."""
import numpy as np
import pytest

from oracle import kv as okv


@pytest.fixture(scope="module")
def S():
    from lora_adapters_gb300 import build, slora

    build.build()
    slora.lib()
    return slora


def test_a_planning_pool_has_no_cache(S):
    pool = S.Pool(64, 256, "f16", [(8, 8)], 1, 1, max_tokens=4)
    with pytest.raises(ValueError):
        S.KVCache(pool, 1, 4, 4, 64, 2, 8)
    with pytest.raises(S.SloraError) as e:
        S.slora_kv_create(pool.handle, 1, 4, 4, 64, 2, 8, 16, 16)
    assert e.value.code == S.ERR_INVALID
    pool.close()


def test_null_handles_are_refused(S):
    for call in (lambda: S.slora_kv_destroy(0), lambda: S.slora_kv_set_rotary(0, 0, 0, []),
                 lambda: S.slora_kv_plan(0, 0, 0, 0, 0, 0, 0, 0, 0),
                 lambda: S.slora_kv_attend(0, S.slora_kv_batch(), 0, 16, 8, 16, 8, 1.0),
                 lambda: S.slora_kv_append(0, S.slora_kv_batch(), 0, 16, 8, 16, 8, 16, 8, 0, 0, 0.0, 16, 8)):
        with pytest.raises(S.SloraError) as e:
            call()
        assert e.value.code == S.ERR_INVALID


def test_oracle_plan_by_hand():
    # blocks of 2; request 0 (row 1) holds 3 tokens and gets 2, request 1 (row 0) is new with 1
    table = np.full((1, 2, 2, 3), -1, np.int32)
    table[0, 0, 1, :2], table[0, 1, 1, :2] = [7, 4], [8, 9]
    got = okv.plan(table, [1, 0], [3, 0], [2, 1], [20, 21, 30, 31], 4, 2, 40)
    assert got["slots"].tolist() == [[[9, 40, 60, -1], [19, 42, 62, -1]]]
    assert got["tok_req"].tolist() == [0, 0, 1, -1] and got["tok_pos"].tolist() == [3, 4, 0, -1]
    assert got["q_start"].tolist() == [0, 2, 3] and got["kv_len"].tolist() == [5, 1]
    assert table[0].tolist() == [[[30, -1, -1], [7, 4, 20]], [[31, -1, -1], [8, 9, 21]]]


def test_oracle_rotation_keeps_scores_of_equal_distance():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 32)), rng.standard_normal((1, 32))
    f = [10000.0 ** (-2 * i / 32) for i in range(16)]
    for inter in (False, True):
        rot = lambda x, p: okv.norm_rotate(x, None, 0.0, p, f, 32, inter, 1.0)
        assert np.isclose((rot(q, 17) * rot(k, 5)).sum(), (rot(q, 1012) * rot(k, 1000)).sum())
        assert np.allclose(rot(q, 0), q)
    y = okv.norm_rotate(q * 100, np.full(32, 2.0), 0.0, 0, f, 0, False, 1.0)
    assert np.isclose((y * y).mean(), 4.0)


def test_oracle_attention_invariants():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 16))
    q = rng.standard_normal((3, 4, 16))
    out = okv.attend(q, k, v, 6, 0.25, 0.0)
    # the first position sees only itself; equal keys average the values; a
    # softcap far above the scores changes nothing
    assert np.allclose(okv.attend(q[:1], k[:1], v[:1], 0, 0.25, 0.0)[0, 3], v[0, 1])
    same = okv.attend(q, np.ones_like(k), v, 6, 0.25, 0.0)
    assert np.allclose(same[1, 0], v[:8, 0].mean(0))
    assert np.allclose(okv.attend(q, k, v, 6, 0.25, 1e6), out, atol=1e-6)


def test_rotary_frequencies_of_each_scaling():
    from lora_adapters_gb300 import rotary

    plain, m = rotary.inv_freq(64)
    assert m == 1.0 and np.allclose(plain, 10000.0 ** (-np.arange(0, 64, 2) / 64))
    assert np.allclose(rotary.inv_freq(64, scaling="linear", factor=4.0)[0], np.array(plain) / 4)
    f, m = rotary.inv_freq(64, scaling="base", factor=8.0)
    assert m == 1.0 and np.isclose(f[0], 1.0) and np.isclose(f[-1], plain[-1] / 8)
    f, m = rotary.inv_freq(64, scaling="parts", factor=8.0, trained_len=4096)
    r = np.array(f) / np.array(plain)
    assert np.isclose(m, 0.1 * np.log(8.0) + 1) and np.isclose(r[0], 1) and np.isclose(r[-1], 1 / 8)
    assert (np.diff(r) <= 1e-12).all()
    turns = 4096 * np.array(plain) / (2 * np.pi)
    assert np.allclose(r[turns > 33], 1) and np.allclose(r[turns < 0.8], 1 / 8)
    for bad in (dict(rot_dim=3), dict(rot_dim=64, factor=0.5), dict(rot_dim=64, scaling="parts"),
                dict(rot_dim=64, scaling="other"), dict(rot_dim=64, base=1.0), dict(rot_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            rotary.inv_freq(**bad)


# ---- caches held in 4 bits ------------------------------------------------------------


def test_4_bit_caches_refuse_what_16_bit_ones_do(S):
    pool = S.Pool(64, 256, "f16", [(8, 8)], 1, 1, max_tokens=4)
    with pytest.raises(ValueError):
        S.KVCache(pool, 1, 4, 4, 64, 2, 8, bits=4)
    for call in (lambda: S.slora_kv_q4_create(pool.handle, 1, 4, 4, 64, 2, 8, 16, 16),
                 lambda: S.slora_kv_q4_array_ints(pool.handle, 1, 4, 4, 64, 2, 8),
                 lambda: S.slora_kv_q4_create(0, 1, 4, 4, 64, 2, 8, 16, 16),
                 lambda: S.slora_kv_q4_array_ints(0, 1, 4, 4, 64, 2, 8),
                 lambda: S.slora_kv_read(0, 0, 1, 16, 16, 16, 8, 32, 8)):
        with pytest.raises(S.SloraError) as e:
            call()
        assert e.value.code == S.ERR_INVALID
    for bits in (2, 8, 5, 0):
        with pytest.raises(ValueError):
            S.KVCache(pool, 1, 4, 4, 64, 2, 8, bits=bits)
    pool.close()


def test_tokens_per_page(S):
    assert S.tokens_per_page(4096, 32, 128) == 1 and S.tokens_per_page(4096, 32, 128, 4) == 3
    assert S.tokens_per_page(5120, 8, 128) == 5 and S.tokens_per_page(5120, 8, 128, 4) == 17
    assert S.tokens_per_page(40, 1, 80, 4) == 1          # 54 bytes, rounded up to 64, in a page of 80
    assert S.tokens_per_page(24, 1, 80, 4) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_oracle_quantiser(dtype):
    """The format by hand, and its bounds on random groups."""
    from oracle import kv_q4 as oq4

    x = np.zeros((1, 32))
    x[0, :6] = [8.0, -8.0, 0.5, -0.5, 0.49, 7.6]
    k, M = oq4.quantise(x, dtype)                        # both signs reach 8: the positive one
    assert M[0, 0] == 8.0 and k[0, :6].tolist() == [8, -7, 1, 0, 0, 8]
    assert oq4.values(k, M, 32)[0, :6].tolist() == [8.0, -7.0, 1.0, 0.0, 0.0, 8.0]
    k, M = oq4.quantise(-x[:, [0, 2, 5] + list(range(6, 32)) + [6, 7, 8]], dtype)
    assert M[0, 0] == -8.0 and k[0, :3].tolist() == [8, 1, 8]
    assert oq4.scale(1.0, dtype) == 1.0 and oq4.scale(1.03, dtype) == 1.0625 and oq4.scale(-33.0, dtype) == -34.0
    assert oq4.scale(1e30, "f16") == 63488.0 and oq4.scale(1e-9, "f16") == 2.0 ** -21 and oq4.scale(0.0, dtype) == 0.0
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 96)) * np.exp(rng.uniform(-6, 6, (40, 1)))
    k, M = oq4.quantise(x, dtype)
    assert k.min() >= -7 and k.max() <= 8 and (np.abs(x).reshape(40, 3, 32).max(-1) <= np.abs(M)).all()
    err, big = np.abs(oq4.values(k, M, 96) - x), np.repeat(np.abs(M), 32, -1)
    same = np.sign(x) == np.sign(np.repeat(M, 32, -1))
    assert (err <= np.where(same, big / 16, big / 8) * (1 + 1e-12)).all()
    held = oq4.values(k, M, 96)                          # eight significant bits: both types hold it
    assert np.array_equal(held, np.round(held / 2.0 ** np.floor(np.log2(np.abs(held) + (held == 0)) - 7))
                          * 2.0 ** np.floor(np.log2(np.abs(held) + (held == 0)) - 7))
    for is_value in (False, True):
        rows = oq4.pack(k[None], M[None], dtype, is_value)
        assert rows.shape == (1, oq4.row_bytes(40, 96)) and np.array_equal(oq4.unpack(rows, 40, 96, dtype, is_value)[0], held)
    # where the header says that codes lie: element 37 = 32 + 5 of a head of 96
    k = np.zeros((1, 1, 96), np.int64) - 7
    k[0, 0, 37] = 8
    M = np.ones((1, 1, 3))
    row = oq4.pack(k, M, dtype, False)[0, :48].view("<u4")
    assert row[0 * 3 + 1] == 15 << (16 * 1 + 4 * 2) and (np.delete(row, 1) == 0).all()
    row = oq4.pack(k, M, dtype, True)[0, :48].view("<u2")
    assert row[1 * 3 + 1] == 15 << (4 * 1) and (np.delete(row, 4) == 0).all()


def test_tokens_per_page_refuses_other_widths(S):
    for bits in (0, 2, 8, 32):
        with pytest.raises(ValueError):
            S.tokens_per_page(4096, 32, 128, bits)
