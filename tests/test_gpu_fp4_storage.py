"""GPU: codes and scales as tensors of their own."""
import io

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from tests import block_cases as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(3, 32), (37, 2880), (2, 300, 512)])
def test_codes_and_scales_share_no_storage(shape):
    """A checkpoint holds them one by one: keeping or saving one of them takes its own bytes alone."""
    codes, scale = M.quantize_fp4(C.randn(C.gen(1), *shape, dtype=torch.bfloat16))
    for t in (codes, scale):
        assert t.untyped_storage().nbytes() == t.numel() and t.storage_offset() == 0
        saved = io.BytesIO()
        torch.save(t, saved)
        assert saved.tell() < t.numel() + 4096
        saved.seek(0)
        assert torch.equal(torch.load(saved), t)
    assert codes.untyped_storage().data_ptr() != scale.untyped_storage().data_ptr()
