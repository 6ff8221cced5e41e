"""Prefill over padded batches: far more rows that belong to no sequence than the pipeline is deep."""
import numpy as np
import pytest
import torch

from window_cases import ALL, WindowCase, pool_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [20000, 60000])
@pytest.mark.parametrize("window", [False, True])
def test_rows_behind_the_last_sequence(cuda_lib, pad, window):
    """paged_attention_prefill gives them zeros and records them, paged_attention_window leaves them; nothing times out."""
    pa = cuda_lib
    pa.device_error_flags(clear=True)
    case = WindowCase(31, [400, 90, 33], [300, 90, 2], ALL, 0, q_heads=8, kv_heads=8, head_dim=64, block_size=16,
                      dtype=torch.bfloat16, tail=pad)
    d, out = case.device(), torch.full(case.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    if window:
        pa.paged_attention_window(**d, window=ALL, scale=case.scale, out=out)
    else:
        pa.paged_attention_prefill(d["q"], d["query_start_loc"], d["k_pool"], d["v_pool"], d["block_table"], d["context_lens"],
                                   case.scale, out=out)
    torch.cuda.synchronize()
    assert pa.device_error_flags(clear=True) == (0 if window else pa.PA_DEVERR_QUERY_LOC)
    rows, ref, spread, size = case.oracle()
    assert (np.abs(out.cpu().double().numpy()[rows] - ref) <= pool_bound(case, ref, spread, size)).all()
    assert (out[392:] == (7 if window else 0)).all()
