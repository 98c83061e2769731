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


def test_4_bit_trace_on_a_planning_pool_takes_fewer_pages():
    sp = small_spec(steps=60)
    sp = dataclasses.replace(sp, attention=True, head_dim=64)
    a, b = (trace.Trace(dataclasses.replace(sp, kv_bits=bits)) for bits in (16, 4))
    ra, rb = a.run(), b.run()
    P = b.spec.kv_tokens_per_page
    assert P > 1 and a.spec.kv_tokens_per_page == 1
    for tr in (a, b):
        need = lambda n: -(-n // tr.spec.kv_tokens_per_page) * sp.kv_pages_per_token
        taken = sorted(tr.kv[rq.kv_handles[0]].shape[0] for rq in tr.running)
        assert taken == sorted(need(rq.prompt + rq.output) for rq in tr.running)
    assert rb.peak_kv_pages * (P - 1) < ra.peak_kv_pages * P
    a.close()
    b.close()
    for bad in (dict(kv_bits=8), dict(kv_bits=4, attention=False)):
        with pytest.raises(ValueError):
            trace.Trace(dataclasses.replace(sp, **bad))
