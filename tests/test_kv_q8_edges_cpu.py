"""What the 8-bit cache's operators write may not lie in itself (refused before any launch; no compute call is made here)."""
import pytest

import block_quantized_routed_gb300 as moe
from tests.test_kv_q8_cpu import INV, append_rc, attn_rc, desc, lib, read_rc, scales  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("kw", [
    dict(sc=scales(k_head_stride=0)), dict(sc=scales(v_page_stride=0)), dict(sc=scales(k_row_stride=0)),
    dict(sc=scales(k_page_stride=31)), dict(sc=scales(v_head_stride=15)), dict(sc=scales(v_row_stride=1, v_head_stride=1)),
    dict(kv=desc(k_head_stride=0)), dict(kv=desc(v_row_stride=64)), dict(kv=desc(k_page_stride=2040)),
    dict(kv=desc(v_head_stride=56)), dict(kv=desc(k_page_stride=0))])
def test_caches_whose_entries_share_memory_are_not_appended_to(lib, kw):  # noqa: F811
    assert append_rc(lib, **kw) == INV


@pytest.mark.parametrize("kw", [dict(oh=0), dict(os=0), dict(oh=56), dict(os=248), dict(os=64, oh=64), dict(os=64, oh=120)])
def test_attention_outputs_that_share_memory_are_refused(lib, kw):  # noqa: F811
    assert attn_rc(lib, **kw) == INV


@pytest.mark.parametrize("kw", [dict(ks=120), dict(vh=56), dict(ks=64, kh=504), dict(vs=0)])
def test_rows_that_share_memory_are_refused(lib, kw):  # noqa: F811
    assert read_rc(lib, **kw) == INV


def test_an_entry_of_one_needs_no_stride(lib):  # noqa: F811
    """A stride over a dimension of one entry is never used; without tokens nothing is looked at."""
    one = dict(num_pages=1, Hkv=1, k_page_stride=0, v_page_stride=0, k_head_stride=0, v_head_stride=0, k_row_stride=64, v_row_stride=64)
    assert append_rc(lib, kv=desc(**one), sc=scales(k_page_stride=0, v_page_stride=0, k_head_stride=0, v_head_stride=0), n=15) == moe.MOE_ERR_WORKSPACE
    assert append_rc(lib, sc=scales(k_head_stride=0), T=0) == 0
