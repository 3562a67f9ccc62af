"""New rows into a paged cache: every slot against a 64-bit reference's place,
and everything that is not a new token's slot bit for bit as it was. Copied
rows are exact; normed and rotated ones equal sdpa_qk_norm_rope's, whose
tolerance test_gpu_norm_rope.py derives, bit for bit."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import scaled_dot_product_02_gb300 as sdpa

pytestmark = pytest.mark.gpu


def batch(seed, new, total, page, hkv, d, dv, order, dtype, pad=0, together=False, hq=None):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    table, pages = ref.make_pages(rng, total, page)
    rows = sum(new) + pad
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    shape = lambda w: (pages, page, hkv, w) if order == "nhd" else (pages, hkv, page, w)  # noqa: E731
    if together:  # pages that hold K and V
        both = n(pages, 2, *shape(d)[1:])
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = n(*shape(d)), n(*shape(dv))
    whole = n(rows, (hq or 0) * d + hkv * (d + dv))
    at = (hq or 0) * d
    s = dict(k=whole[:, at:at + hkv * d].unflatten(1, (hkv, d)), v=whole[:, at + hkv * d:].unflatten(1, (hkv, dv)),
             kc=kc, vc=vc, table=table, cu=cu, lens=np.array(total, dtype=np.int32), page=page, order=order)
    if hq:
        s["q"] = whole[:, :at].unflatten(1, (hq, d))
    s["dev"] = (torch.from_numpy(table).cuda(), torch.from_numpy(s["lens"]).cuda(), torch.from_numpy(cu).cuda())
    return s


def expected(s, k_rows, v_rows):
    row, page, slot, _, _ = ref.token_places(s["cu"], s["lens"], s["page"], s["table"])
    kc, vc = s["kc"].clone(), s["vc"].clone()
    row, page, slot = (torch.from_numpy(a).cuda() for a in (row, page, slot))
    for cache, x in ((kc, k_rows), (vc, v_rows)):
        (cache if s["order"] == "nhd" else cache.transpose(1, 2))[page, slot] = x[row]
    return kc, vc


BATCHES = [([1] * 5, [1, 17, 16, 33, 1000]), ([0, 3, 0, 70, 1], [0, 3, 40, 129, 64]), ([1], [1]), ([257], [257]),
           ([2] * 70, list(range(2, 72)))]


@pytest.mark.parametrize("new,total", BATCHES)
@pytest.mark.parametrize("d,dv,page,order,together", [(128, 128, 16, "nhd", False), (256, 256, 48, "hnd", True),
                                                      (192, 128, 32, "hnd", False), (512, 512, 256, "nhd", True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_copied_rows(new, total, d, dv, page, order, together, dtype):
    s = batch(1, new, total, page, 3, d, dv, order, dtype, pad=4, together=together)
    kc, vc = expected(s, s["k"], s["v"])
    got = sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], *s["dev"], cache_layout=order)
    assert got is None and torch.equal(s["kc"], kc) and torch.equal(s["vc"], vc)
    assert sdpa.sdpa_last_launch_count() == 1
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("new,total", BATCHES)
@pytest.mark.parametrize("d,dv,rot,inter", [(128, 128, 128, False), (192, 128, 64, False), (256, 256, 256, True),
                                            (512, 512, 128, False), (128, 128, 0, False)])
def test_normed_and_rotated_on_the_way(new, total, d, dv, rot, inter):
    s = batch(2, new, total, 16, 2, d, dv, "nhd", torch.bfloat16, pad=3, hq=6)
    wq, wk = (1 + 0.2 * torch.randn(2, d, device="cuda")).bfloat16()
    table = ref.angles_table(1000, rot)
    table = None if table is None else table.cuda()
    row, _, _, pos, _ = ref.token_places(s["cu"], s["lens"], 16, s["table"])
    where = torch.zeros(s["k"].shape[0], dtype=torch.int32)
    where[torch.from_numpy(row)] = torch.from_numpy(pos).int()
    for positions in (None, (where.cuda() * 7 + 3) % 1000):
        at = where.cuda() if positions is None else positions
        q_ref, k_ref = sdpa.sdpa_qk_norm_rope(s["q"], s["k"], wq, wk, table, at, interleaved=inter)
        kc, vc = expected(s, k_ref, s["v"])
        q_out = torch.full_like(q_ref, 5.0)
        got = sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], *s["dev"], q=s["q"], q_weight=wq, k_weight=wk,
                                     cos_sin=table, positions=positions if rot else None, interleaved=inter, q_out=q_out)
        assert got is q_out and torch.equal(s["kc"], kc) and torch.equal(s["vc"], vc)
        live = torch.zeros(q_out.shape[0], dtype=torch.bool)
        live[torch.from_numpy(row)] = True
        live = live.cuda()
        assert torch.equal(q_out[live], q_ref[live]) and bool((q_out[~live] == 5).all())
    assert sdpa.sdpa_get_device_error() == 0


def test_bad_metadata_is_recorded_and_nothing_of_it_written():
    s = batch(3, [2, 3, 1], [20, 33, 5], 16, 2, 128, 128, "nhd", torch.bfloat16)
    table, lens, cu = s["dev"]
    pages = s["kc"].shape[0]
    for bad, code in ((pages, 10), (-1, 10), (2 ** 31 - 1, 10)):
        t = table.clone()
        t[1, 2] = bad  # sequence 1's positions 30..32: the last one is on this page
        kept = s["kc"].clone(), s["vc"].clone()
        kc, vc = expected(s, s["k"], s["v"])
        row, page, slot, pos, b = ref.token_places(s["cu"], s["lens"], 16, s["table"])
        skip = (b == 1) & (pos >= 32)
        i, j = torch.from_numpy(page[skip]).cuda(), torch.from_numpy(slot[skip]).cuda()
        kc[i, j], vc[i, j] = kept[0][i, j], kept[1][i, j]
        sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], t, lens, cu)
        assert sdpa.sdpa_get_device_error() == code
        assert torch.equal(s["kc"], kc) and torch.equal(s["vc"], vc)
        s["kc"].copy_(kept[0])
        s["vc"].copy_(kept[1])
    # a length shorter than its new tokens, and one past the table
    for n in (1, 49):
        short = lens.clone()
        short[1] = n
        sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], table, short, cu)
        assert sdpa.sdpa_get_device_error() in (6, 10)
    # sequences that end behind the tensors' rows
    sdpa.sdpa_paged_append(s["k"][:4], s["v"][:4], s["kc"], s["vc"], table, lens, cu)
    assert sdpa.sdpa_get_device_error() == 6
    assert sdpa.sdpa_get_device_error() == 0


def test_captured_replays_follow_the_lengths():
    s = batch(4, [1, 1, 1], [9, 31, 64], 16, 2, 128, 128, "nhd", torch.bfloat16)
    table, lens, cu = s["dev"]
    full = torch.arange(3 * 6, device="cuda", dtype=torch.int32).view(3, 6)
    kc, vc = torch.zeros(18, 16, 2, 128, device="cuda").bfloat16(), torch.zeros(18, 16, 2, 128, device="cuda").bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdpa.sdpa_paged_append(s["k"], s["v"], kc, vc, full, lens, cu)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(lens.tolist()):
            assert torch.equal(kc.view(3, 96, 2, 128)[b, n - 1], s["k"][b])
            assert torch.equal(vc.view(3, 96, 2, 128)[b, n - 1], s["v"][b])
        lens += 1
    assert int((kc != 0).any(-1).any(-1).sum()) == 9


@pytest.mark.parametrize("rot", [0, 128])
def test_every_access_is_inside_the_buffers(rot):
    s = batch(5, [0, 3, 70, 1], [12, 3, 129, 64], 48, 2, 128, 128, "hnd", torch.float16, pad=2, hq=4)
    kw = {}
    if rot:
        kw = dict(q=s["q"], q_weight=torch.ones(128, device="cuda").half(), k_weight=torch.ones(128, device="cuda").half(),
                  cos_sin=ref.angles_table(200, rot).cuda())
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], *s["dev"], cache_layout="hnd", **kw)
        assert sdpa.sdpa_debug_address_report()[0] == 0
        assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("given", [False, True])
def test_a_token_whose_position_has_no_angles_is_skipped_whole(given):
    s = batch(4, [3, 2], [22, 9], 16, 2, 128, 128, "nhd", torch.bfloat16, hq=4)  # positions 19 to 21, 7 and 8
    w, table = torch.ones(128, device="cuda").bfloat16(), ref.angles_table(20, 128).cuda()
    positions = torch.tensor([19, 20, 21, 7, 8], dtype=torch.int32, device="cuda")
    _, k_ref = sdpa.sdpa_qk_norm_rope(s["q"], s["k"], w, w, table, positions.clamp(max=19))
    kept = s["kc"].clone(), s["vc"].clone()
    kc, vc = expected(s, k_ref, s["v"])
    _, page, slot, _, _ = ref.token_places(s["cu"], s["lens"], 16, s["table"])
    i, j = torch.from_numpy(page[1:3]).cuda(), torch.from_numpy(slot[1:3]).cuda()
    kc[i, j], vc[i, j] = kept[0][i, j], kept[1][i, j]
    q_out = torch.full_like(s["q"], 5.0, memory_format=torch.contiguous_format)
    sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], *s["dev"], q=s["q"], q_weight=w, k_weight=w, cos_sin=table,
                           positions=positions if given else None, q_out=q_out)
    assert sdpa.sdpa_get_device_error() == 10
    assert torch.equal(s["kc"], kc) and torch.equal(s["vc"], vc)
    assert bool((q_out[1:3] == 5).all()) and bool((q_out[[0, 3, 4]] != 5).any())


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("at", [1, 2, 3, 4])
@pytest.mark.parametrize("v_first", [False, True])
@pytest.mark.parametrize("hkv", [1, 3])
def test_caches_that_interleave_at_every_level(order, at, v_first, hkv):
    """K and V in turn by page, by the outer and the inner one of slot and head, and side by side in a row."""
    s = batch(7, [3, 0, 20], [30, 5, 61], 16, hkv, 128, 128, order, torch.bfloat16, pad=1)
    shape = list(s["kc"].shape)
    both = torch.randn(*shape[:at], 2, *shape[at:], device="cuda").bfloat16()
    if at == 4:  # [..., 2 x width]
        both = torch.randn(*shape[:3], 256, device="cuda").bfloat16()
        k, v = both[..., :128], both[..., 128:]
    else:
        k, v = both.select(at, 0), both.select(at, 1)
    s["kc"], s["vc"] = (v, k) if v_first else (k, v)
    kc, vc = expected(s, s["k"], s["v"])
    sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], *s["dev"], cache_layout=order)
    assert torch.equal(s["kc"], kc) and torch.equal(s["vc"], vc)
    assert sdpa.sdpa_get_device_error() == 0
    with pytest.raises(sdpa.SdpaError, match="OVERLAP"):
        sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["kc"], *s["dev"], cache_layout=order)
