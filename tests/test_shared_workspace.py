"""What a decode behind shared prefixes asks for as workspace: the expanded records are bounded whatever the tables' widths."""
import ctypes as C

import pytest

from sparse_mla_decode_paged_gb300._native import SmlaSharedDims

TILE_BYTES = 128 * 576 * 2                                  # a tile of 128 positions in fp16
SMS = 152


def size(lib, requests, heads, prefixes, prefix_pages, own_pages):
    d = SmlaSharedDims(requests, heads, 64, own_pages, 512, 64, 1 << 20, 1, prefixes, prefix_pages)
    n = C.c_size_t(0)
    return lib.sparse_mla_shared_workspace_size(d, SMS, C.byref(n)), n.value


def beside(requests, heads):
    """Bytes for anything but the expansion, at most: two fp32 results per row, the dense kernel's and the pairs' parts of
    128 and 64 rows per CTA, two lse each, and 64 MiB for places and exponents."""
    return requests * heads * 2 * 513 * 4 + 2 * (2 * SMS * 128 * 513 * 4) + (64 << 20)


@pytest.mark.parametrize("requests,heads,prefixes", [(256, 128, 1), (1024, 64, 2), (4096, 16, 1), (64, 128, 64), (8, 16, 1)])
@pytest.mark.parametrize("prefix_pages", [16, 512, 20000, 58254])
@pytest.mark.parametrize("own_pages", [1, 16, 1000, 20000])
def test_the_expansion_is_bounded(lib, requests, heads, prefixes, prefix_pages, own_pages):
    status, n = size(lib, requests, heads, prefixes, prefix_pages, own_pages)
    assert status == 0
    assert n <= (5 << 30) + beside(requests, heads)


def test_wide_tables_of_the_requests_are_not_refused(lib):
    # 2^29 tiles and more of the requests' own, which the dense kernel takes
    status, n = size(lib, 65535, 16, 1, 512, 17000)
    assert status == 0
    assert n <= 512 // 2 * TILE_BYTES + beside(65535, 16)
