"""The 8-bit paged cache: what is told of a call without rows."""
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.q8_ref import E4M3, Q8Cache, new_ws, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def test_keys_without_rows_are_told():
    """No rows at all: every key lies outside them."""
    c = Q8Cache([20, 0], 2, 64, 16, E4M3)
    first = torch.tensor([0, 20], dtype=torch.int32).cuda()
    out = torch.empty(0, 2, 64, device="cuda")
    for lens, want in (([20, 0], moe.MOE_ERR_DEVICE_BOUNDS), ([0, 3], moe.MOE_ERR_DEVICE_BOUNDS), ([0, -1], moe.MOE_ERR_DEVICE_BOUNDS),
                       ([0, 0], 0)):
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        ws = new_ws()
        moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, c.gtable, c.kv_len, first, out, out.clone(), ws)
        assert status(ws) == want, lens
