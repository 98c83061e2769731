"""Run in a process of its own with SLORA_DEBUG=1 (tests/test_gpu_kv_q4_edges.py): the
4-bit key-value cache in the SLORA_DEBUG build.

A step computes as the release build does; a slot, a table row or a token index planted
in a batch's arrays is caught before it addresses memory (SLORA_ERR_DEVICE_ASSERT), in
append and in both attention kernels; planned again, the step is right again.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from lora_adapters_gb300 import slora  # noqa: E402
from tests.test_gpu_kv_q4 import Setup, _attend  # noqa: E402


def main() -> int:
    assert slora.DEBUG and slora.LIB_PATH.endswith("libslora_debug.so"), slora.LIB_PATH
    s = Setup(slora, [900, 30, 200], [1, 40, 1], 4, 2, 64, 320, "f16", T=50)
    s.oracle_plan()
    held = s.fill()
    b, q, out = _attend(s, held)
    w = s.hq * s.d
    k = s.randn(s.T, s.hkv * s.d)
    keep = s.pool.buffer.clone()
    for bad in (s.num_pages * s.P, 1 << 30):
        for kind in (0, 1):
            old = b.slots[0, kind, 5].clone()
            b.slots[0, kind, 5] = bad
            s.kv.append(b, 0, q, k, k, q_out=torch.empty_like(q))
            assert s.pool.status() == slora.ERR_DEVICE_ASSERT, (bad, kind)
            b.slots[0, kind, 5] = old
    s.pool.buffer.copy_(keep)
    req = s.kv.arrays[: 4 * 3].view(3, 4)        # {first token, new tokens, tokens held, table row}
    for r in (0, 1):                             # a decode request, a chunk
        for field, values in ((3, (s.table.shape[2], -1)), (0, (s.T, s.T + 7, -50))):
            for bad in values:
                old = req[r, field].clone()
                req[r, field] = bad
                s.kv.attend(b, 0, q, out[:, :w])
                assert s.pool.status() == slora.ERR_DEVICE_ASSERT, (r, field, bad)
                req[r, field] = old
    _attend(s, held)
    s.close()
    print("debug build OK")
    return 0


if __name__ == "__main__":
    sys.exit(main())
