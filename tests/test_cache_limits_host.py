"""The longest sequence a paged cache may describe (no GPU; the pointers are never followed): the decode
kernels round a length up to units of 64 keys in 32 bits."""
import ctypes

import pytest

import context_blockwise_attention_step_gb300 as ra
from context_blockwise_attention_step_gb300 import _abi

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ra.build()


def cache(max_pages, page):
    c = _abi.RaPagedCache()
    for k, v in dict(dtype=_abi.RA_BF16, hkv=2, head_dim=128, page_size=page, n_pages=8, n_seqs=3, max_pages=max_pages,
                     table_stride=max_pages, page_stride=page * 256, slot_stride=256, head_stride=128, k_pages=FAKE,
                     v_pages=FAKE, block_table=FAKE).items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("max_pages,page", [(2 ** 27 - 1, 16), (1, 2 ** 31 - 1), (2 ** 31 - 1, 1), (1, 2 ** 31 - 63)])
def test_longer_caches_are_refused(max_pages, page):
    L, c = _abi.lib(), cache(max_pages, page)
    assert L.ra_paged_workspace_bytes(c, 8) == 0
    assert L.ra_paged_attn_decode(c, 8, 0.0, 0, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == _abi.RA_ERR_UNSUPPORTED
    assert L.ra_kv_cache_append(c, None, 0.0, 3, 8, FAKE, 1024, FAKE, 256, FAKE, 256, None, None, FAKE, None, 512,
                                None) == _abi.RA_ERR_UNSUPPORTED


def test_the_longest_is_not():
    for max_pages, page in ((2 ** 25 - 1, 64), (1, 2 ** 31 - 64), (2 ** 31 - 64, 1)):
        assert _abi.lib().ra_paged_workspace_bytes(cache(max_pages, page), 8) > 0
