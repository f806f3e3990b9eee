"""Rows narrower than a wave's columns with as many choices as there can be:
most lanes hold a choice and none of the row."""
import pytest
import torch

from tests import expertskit as kit
from tests.routekit import log
from tests.test_gpu_experts_rows import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,topk,width,count", [(3, 64, 1, 64), (40, 64, 8, 64), (70, 63, 9, 40), (9, 64, 64, 30),
                                                   (33, 64, 520, 64)])
def test_more_choices_than_lanes_with_columns(rows, topk, width, count, dtype):
    log(f"narrow {rows}x{topk}x{width} {dtype}")
    check(kit.RowsCase(rows, topk, width, 64, count, dtype, seed=width))
