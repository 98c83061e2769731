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
