"""Reads of many rows of an 8-bit paged cache on both sides of the rules that choose how
many tokens a warp takes; every value is exact. The sequences share a few pages, so
that the rows are many and the cache is small."""
import numpy as np
import pytest
import torch

import fp8_ref
import scaled_dot_product_02_gb300 as sdpa

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("rows", [39999, 40003])
@pytest.mark.parametrize("hkv,d", [(8, 128), (2, 512), (9, 128), (16, 128), (8, 256), (5, 512), (7, 192)])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
def test_many_rows(rows, hkv, d, order):
    """256 vectors of 8 values a token and more, up to 40000 rows and above."""
    page, pages, dv = 64, 7, 128 if d == 192 else d
    rng, g = np.random.default_rng(rows + d), torch.Generator().manual_seed(hkv)
    kc, ks = fp8_ref.quantise(torch.randn(pages, page, hkv, d, generator=g), BF)
    vc, vs = fp8_ref.quantise(torch.randn(pages, page, hkv, dv, generator=g), BF)
    lens = np.array([rows // 2, rows - rows // 2 + 70], dtype=np.int32)  # the second one's last keys alone
    cu = np.array([0, rows // 2, rows], dtype=np.int32)
    table = rng.integers(0, pages, (2, -(-int(lens.max()) // page))).astype(np.int32)
    dev = [(x if order == "nhd" else x.transpose(1, 2).contiguous()).cuda() for x in (kc, vc, ks, vs)]
    k, v = sdpa.sdpa_paged_read_fp8(*dev, *(torch.from_numpy(x).cuda() for x in (table, lens, cu)), cache_layout=order,
                                    rows=rows + 2, dtype=BF, k_out=torch.full((rows + 2, hkv, d), 3.0, dtype=BF, device="cuda"))
    at = np.concatenate([np.arange(rows // 2), np.arange(70, lens[1])])
    seq = np.repeat([0, 1], [rows // 2, rows - rows // 2])
    where = torch.from_numpy(table[seq, at // page].astype(np.int64)).cuda(), torch.from_numpy(at % page).cuda()
    for got, codes, scale in ((k, kc, ks), (v, vc, vs)):
        want = fp8_ref.decode(codes, scale).to(BF).cuda()  # exact in the type
        assert torch.equal(got[:rows], want[where])
    assert bool((k[rows:] == 3).all()) and sdpa.sdpa_get_device_error() == 0
