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
