"""What the binding of the step calls refuses, one change at a time to calls that succeed, by type and message."""
import numpy as np
import pytest
import torch

from pagedattention_kv_cache_paged_gb300 import _abi
from tree_cases import TreeCase

pytestmark = pytest.mark.gpu


def tree_args():
    case = TreeCase(1, [4, 40], [2, 3], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=torch.float32)
    return case.device()


def tables_args():
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return dict(history_lens=i32([4, 17]), new_lens=i32([2, 3]), block_table=i32([[0, -1, -1], [1, 2, -1]]),
                block_counts=i32([1, 2]), free_blocks=i32([3, 4, 5]), free_state=i32([3, 0]), block_size=16, num_blocks=6,
                parents=i32([-1, 0, -1, 0, 0]))


def accept_args():
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((2, 6, 16, 2, 64), device="cuda") for _ in range(2))
    return dict(k_pool=k, v_pool=v, accepted=i32([[0, 2], [1, 0]]), accepted_lens=i32([2, 1]), history_lens=i32([4, 17]),
                block_table=i32([[0, -1, -1], [1, 2, -1]]))


CALLS = {"paged_attention_tree": tree_args, "build_block_tables": tables_args, "paged_kv_accept": accept_args}
TENSORS = [(call, name) for call, names in
           (("paged_attention_tree", "q query_start_loc tree_mask k_pool v_pool block_table context_lens"),
            ("build_block_tables", "history_lens new_lens block_table block_counts free_blocks free_state parents"),
            ("paged_kv_accept", "k_pool v_pool accepted accepted_lens history_lens block_table"))
           for name in names.split()]


@pytest.mark.parametrize("call", list(CALLS))
def test_the_calls_succeed_as_they_are(cuda_lib, call):
    cuda_lib.device_error_flags(clear=True)
    getattr(cuda_lib, call)(**CALLS[call]())
    torch.cuda.synchronize()
    assert cuda_lib.device_error_flags() == 0


@pytest.mark.parametrize("call,name", TENSORS)
def test_what_is_no_tensor(cuda_lib, call, name):
    args = CALLS[call]()
    for wrong in (args[name].cpu().numpy(), args[name].tolist(), 7):
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            getattr(cuda_lib, call)(**{**args, name: wrong})


@pytest.mark.parametrize("call,name", TENSORS)
def test_tensors_of_another_type_or_place(cuda_lib, call, name):
    args = CALLS[call]()
    with pytest.raises((TypeError, ValueError), match="must be torch|of one dtype|unsupported dtype"):
        getattr(cuda_lib, call)(**{**args, name: args[name].to(torch.float64)})
    with pytest.raises(ValueError, match="must be a CUDA tensor|is on cpu|is on cuda"):
        getattr(cuda_lib, call)(**{**args, name: args[name].cpu()})


def strided(t):
    return torch.stack([t, t], -1)[..., 0]


@pytest.mark.parametrize("call,change,match", [
    ("paged_attention_tree", lambda a: dict(q=a["q"][0]), r"q must be \[total_q"),
    ("paged_attention_tree", lambda a: dict(q=a["q"][:, :, :32].contiguous()), r"q must be \[total_q"),
    ("paged_attention_tree", lambda a: dict(q=strided(a["q"])), "(q|out) must be contiguous"),
    ("paged_attention_tree", lambda a: dict(tree_mask=a["tree_mask"][:3]), r"tree_mask must be \[total_q"),
    ("paged_attention_tree", lambda a: dict(tree_mask=a["tree_mask"][:, :0]), r"tree_mask must be \[total_q"),
    ("paged_attention_tree", lambda a: dict(tree_mask=strided(a["tree_mask"])), "tree_mask must be contiguous"),
    ("paged_attention_tree", lambda a: dict(block_table=a["block_table"][:1]), r"block_table must be \[batch"),
    ("paged_attention_tree", lambda a: dict(block_table=strided(a["block_table"])), r"block_table must be \[batch"),
    ("paged_attention_tree", lambda a: dict(query_start_loc=a["query_start_loc"][:2]), r"query_start_loc must be \[3\]"),
    ("paged_attention_tree", lambda a: dict(context_lens=a["context_lens"][:1]), r"block_table must be \[batch"),
    ("paged_attention_tree", lambda a: dict(v_pool=a["v_pool"][:2]), "k_pool and v_pool must both be"),
    ("paged_attention_tree", lambda a: dict(k_pool=strided(a["k_pool"])), "k_pool: each block must be contiguous"),
    ("paged_attention_tree", lambda a: dict(out=a["q"][:2]), r"out must be \[5, 4, 64\]"),
    ("paged_attention_tree", lambda a: dict(out=strided(a["q"])), "out must be contiguous"),
    ("paged_attention_tree", lambda a: dict(workspace=torch.zeros((64, 2), dtype=torch.uint8, device="cuda")[:, 0]), "workspace must be contig"),
    ("build_block_tables", lambda a: dict(parents=None), "num_tokens is needed"),
    ("build_block_tables", lambda a: dict(new_lens=a["new_lens"][:1]), r"new_lens must be \[2\]"),
    ("build_block_tables", lambda a: dict(block_table=a["block_table"].t()), r"block_table must be \[batch"),
    ("build_block_tables", lambda a: dict(block_counts=strided(a["block_counts"])), "block_counts must be contiguous"),
    ("build_block_tables", lambda a: dict(free_state=a["free_state"][:1]), r"free_state must be \[2\]"),
    ("build_block_tables", lambda a: dict(num_tokens=4), r"parents must be \[4\]"),
    ("paged_kv_accept", lambda a: dict(k_pool=a["k_pool"][0]), "k_pool and v_pool must both be"),
    ("paged_kv_accept", lambda a: dict(accepted=a["accepted"][:1]), r"accepted must be \[batch"),
    ("paged_kv_accept", lambda a: dict(accepted=a["accepted"].t()), r"accepted must be \[batch"),
    ("paged_kv_accept", lambda a: dict(history_lens=a["history_lens"][:1]), r"history_lens must be \[2\]"),
    ("paged_kv_accept", lambda a: dict(block_table=a["block_table"][0]), r"block_table must be \[batch"),
    ("paged_kv_accept", lambda a: dict(v_pool=a["v_pool"].repeat_interleave(2, 0)[::2]), "equally far apart"),
])
def test_tensors_of_another_layout(cuda_lib, call, change, match):
    args = CALLS[call]()
    with pytest.raises(ValueError, match=match):
        getattr(cuda_lib, call)(**{**args, **change(args)})


def test_the_arrays_of_another_step(cuda_lib):
    pa, args = cuda_lib, tables_args()
    out = pa.build_block_tables(**args)
    for change, match in ((dict(tree_mask=None), "out.tree_mask must be"), (dict(slot_mapping=out.slot_mapping[:3]), "must be"),
                          (dict(context_lens=out.context_lens[:1]), r"context_lens must be \[2\]"),
                          (dict(positions=out.positions.long()), "positions must be torch.int32")):
        with pytest.raises((ValueError, TypeError), match=match):
            pa.build_block_tables(**args, out=out._replace(**change))
    for name in ("query_start_loc", "context_lens", "slot_mapping", "positions", "tree_mask"):
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            pa.build_block_tables(**args, out=out._replace(**{name: [1]}))


def test_workspace_sizes(cuda_lib):
    """Positive where contexts are split, 0 for each size that the call refuses."""
    lib, pa = cuda_lib.load_library(), cuda_lib
    good = [2, 8, 4, 512, 16, 8, 2, 64, pa.PA_BF16]
    assert lib.paged_attention_tree_workspace_size(*good, None) > 0
    assert pa.tree_workspace_size(2, 8, 4, 512, 16, 8, 2, 64, torch.bfloat16) > 0
    for i in range(8):
        for wrong in (0, -1):
            bad = list(good)
            bad[i] = wrong
            assert lib.paged_attention_tree_workspace_size(*bad, None) == 0, (i, wrong)
    for i, wrong in ((5, 7), (5, 64), (7, 96), (8, 9)):  # heads, head_dim, type
        bad = list(good)
        bad[i] = wrong
        assert lib.paged_attention_tree_workspace_size(*bad, None) == 0, (i, wrong)


def test_workspace_sizes_of_refused_blocks_and_kernels(cuda_lib):
    pa = cuda_lib
    size = lambda S, dtype, kernel: pa.tree_workspace_size(2, 8, 4, 512, S, 8, 2, 64, dtype, kernel=kernel)
    for S in (3, 12, 24, 512):
        assert size(S, torch.bfloat16, 0) == 0, S
    assert size(8, torch.bfloat16, 0) > 0 and size(8, torch.bfloat16, 2) == 0
    assert size(16, torch.float32, 0) > 0 and size(16, torch.float32, 2) == 0
    assert size(16, torch.bfloat16, 2) > 0


@pytest.mark.parametrize("change,status", [
    (dict(kernel=2), "EUNSUPPORTED"), (dict(kernel=3), "EINVAL"), (dict(kernel=-1), "EINVAL"),
    (dict(partition_tokens=-1), "EINVAL"), (dict(partition_tokens=2 ** 30 + 1), "EINVAL"), (dict(scale=0), "EINVAL"),
    (dict(scale=-1.0), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(max_nodes=0), "EINVAL"),
])
def test_options_that_the_library_refuses(cuda_lib, change, status):
    with pytest.raises(cuda_lib.PagedAttnError) as e:
        cuda_lib.paged_attention_tree(**{**tree_args(), **change})
    assert e.value.status == getattr(_abi, "PA_" + status)


def test_options_as_other_numbers(cuda_lib):
    """What numpy and torch hold numbers in."""
    pa, args = cuda_lib, tree_args()
    want = pa.paged_attention_tree(**args, scale=0.25, max_nodes=4)
    for scale in (np.float32(0.25), torch.tensor(0.25)):
        assert torch.equal(pa.paged_attention_tree(**args, scale=scale, max_nodes=np.int64(4)), want)
