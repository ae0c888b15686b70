"""The serving operators' refusals at the edges, without a GPU."""
import pytest
import torch

import event_tensor_task_b200 as mk
from test_serve_host import INVALID, append_args, calls, tensors


@pytest.mark.parametrize("row,head,page", [
    (64, 64, 2048),          # row r + 1 of a head is row r of the next
    (64, 1024, 64),          # and of the next page
    (64, 512, 2048),         # half of a head's rows
    (128, 64, 1024),         # heads inside rows, pages inside the rows of a page
    (64, 1024, 1024),        # a page on the second head of the page before
    (1 << 37, 64, 1 << 37),
    (4096, 1 << 37, 1 << 37),
])
def test_append_refuses_pools_whose_rows_overlap(row, head, page):
    a = append_args()
    a.pages.row_stride, a.pages.head_stride, a.pages.page_stride = row, head, page
    with pytest.raises(mk.MkError, match="overlap") as e:
        mk.mk_append_kv(a)
    assert e.value.status == INVALID


@pytest.mark.parametrize("row,head,page", [
    (64, 1024, 2048), (128, 64, 2048), (64, 4096, 1024), (512, 256, 64), (256, 4096, 64), (512, 64, 128), (80, 1280, 4096),
    (128, 2048, 64),         # two pools of one buffer, row by row
])
def test_append_takes_pools_in_any_order_of_their_dimensions(row, head, page):
    a = append_args()
    a.pages.row_stride, a.pages.head_stride, a.pages.page_stride = row, head, page
    a.pages.n_pages = 2 if page == 64 and head == 2048 else 4
    a.rope_theta = 0.5  # refused for this, which is looked at after the pool
    with pytest.raises(mk.MkError, match="rope_theta"):
        mk.mk_append_kv(a)


@pytest.mark.parametrize("name", ["prompt", "paged"])
@pytest.mark.parametrize("scale", [1e-50, 5e-324, 0.0, float("nan")])
def test_a_scale_that_fp32_rounds_to_zero_is_refused(name, scale):
    """(it would become the default scale)"""
    with pytest.raises(mk.MkError, match="scale") as e:
        calls(tensors(), scale=scale)[name]()
    assert e.value.status == INVALID


def test_causal_without_a_truth_value_raises_its_own_error():
    x = tensors()
    with pytest.raises(RuntimeError, match="ambiguous"):
        mk.prompt_attention(x["q"], x["k"], x["k"], x["cu"], causal=torch.ones(2))
    none = x["q"][:0]
    with pytest.raises(RuntimeError, match="ambiguous"):
        mk.prompt_attention(none, none[:, :2], none[:, :2], torch.zeros(1, dtype=torch.int32), causal=torch.ones(2))
