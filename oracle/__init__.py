"""CPU oracle for paged KV-cache attention.  TEST INFRASTRUCTURE ONLY: imported by the tests,
``__graft_entry__.smoke()`` and the CPU-baseline leg of ``bench.py``, never by the library."""
from .paged_oracle import (  # noqa: F401
    causal_attention_contiguous,
    copy_blocks,
    gather_history,
    history_slots,
    lse_merge,
    online_softmax_attention,
    paged_decode,
    paged_decode_rows,
    paged_kv_write,
    paged_prefill,
    partition_partials,
    prefill_query_bound,
    repeat_kv,
    slot_of,
    softmax_attention,
    to_f64,
    to_int,
    transfer_blocks,
)
from . import tree_oracle as tree  # noqa: F401
