"""Attention over an 8-bit paged cache where the scales are at the end of their range."""
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.q8_ref import E4M3, INT8, Q8Cache
from tests.test_gpu_attn_q8 import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("D", [64, 128, 256, 80])
def test_values_whose_scales_are_all_tiny(fmt, D):
    """Scales from 2^-126, the least that appending writes, to 2^-115: the results are normal numbers of bf16.  In one
    CTA, in parts that several join, and with a few keys of no value that hold most of the weight."""
    for lens, q_lens, heads in (([70, 9], [3, 1], 4), ([5000], [1], 8)):
        c = Q8Cache(lens, 1, D, 16, fmt, seed=D)
        g = torch.Generator().manual_seed(5)
        c.vs.copy_(torch.pow(2.0, -126 + 11 * torch.rand(c.vs.shape, generator=g)))
        c.gvs.copy_(c.vs)
        check(c, q_lens, heads)
        p0 = int(c.table[0, 0])
        c.vs[p0, :4] = 0.0
        c.ks[p0, :4] *= 8.0
        c.gvs.copy_(c.vs)
        c.gks.copy_(c.ks)
        check(c, q_lens, heads, seed=1)
