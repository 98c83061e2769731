"""CPU test of the serving trace with attention, on a planning pool."""
import dataclasses

import pytest

from lora_adapters_gb300 import trace
from tests.test_trace import small_spec


def test_attention_trace_on_a_planning_pool_keeps_the_pool_calls():
    """Attention changes no page: the same calls with and without it, a table
    row per running request and every row back at the end."""
    sp = small_spec(steps=60)
    plain = trace.Trace(sp)
    a = plain.run()
    with_kv = trace.Trace(dataclasses.replace(sp, attention=True, head_dim=64))
    b = with_kv.run()
    assert [o[:2] for o in a.ops] == [o[:2] for o in b.ops] and a.tokens == b.tokens
    assert "attention_ms" not in a.summary()
    rows = sorted(with_kv.free_rows + [rq.row for rq in with_kv.running])
    assert rows == list(range(sp.max_running))
    with pytest.raises(ValueError):
        trace.Trace(dataclasses.replace(sp, attention=True, head_dim=48))
    with pytest.raises(ValueError):
        trace.Trace(dataclasses.replace(sp, attention=True, kv_pages_per_token=2 * sp.layers + 1))
    plain.close()
    with_kv.close()
