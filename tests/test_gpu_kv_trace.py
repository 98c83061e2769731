"""GPU test of the serving trace with attention: a traced layer against the oracle."""
import dataclasses

import numpy as np
import pytest
import torch

from lora_adapters_gb300 import trace
from tests.test_trace import small_spec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("probe_step,layer", [(25, 0), (60, 1)])
def test_traced_attention_matches_oracle(probe_step, layer):
    """The trace with attention: at the probed step and layer, the o
    projection's input against the fp64 attention over the keys and values the
    block table names in the pool, for every request of the batch (prompts in
    chunks and decode tokens side by side)."""
    from oracle import kv as okv

    sp = dataclasses.replace(small_spec(steps=probe_step + 2), attention=True, head_dim=64)
    tr = trace.Trace(sp, device=torch.device("cuda", 0), probe_step=probe_step, probe_layer=layer)
    res = tr.run()
    pr = tr.probe
    assert pr is not None and res.attention_ms["kv_attend"] > 0 and res.gpu_ms > 0
    d, heads = sp.head_dim, sp.H // sp.head_dim
    pages = pr["pages"].double().numpy().reshape(-1, heads, d)
    q, got = (pr[k].double().numpy().reshape(-1, heads, d) for k in ("q_rot", "x_o"))
    u = 2.0 ** -11 if sp.dtype == "f16" else 2.0 ** -8
    t0 = 0
    for row, ctx, n in pr["step_plan"]:
        keys, vals = (pages[pr["table"][j, row, :ctx + n]] for j in (0, 1))
        want = okv.attend(q[t0:t0 + n], keys, vals, ctx, d ** -0.5, 0.0)
        tol = u * np.abs(want) + (2.0 ** -12 + u) * np.abs(vals).max((0, 2))[None, :, None]
        assert (np.abs(got[t0:t0 + n] - want) <= tol).all(), (row, ctx, n)
        t0 += n
    assert t0 == pr["ids"].shape[0]
    tr.close()
