"""Each checked access of the 8-bit cache's calls and of rotations with several axes,
by itself: with every extent 16 bytes short a call skips what lies in the last 16
bytes of a buffer, and nothing else. The lengths and the block table lie inside
another input's extent, or end in entries that nothing needs, so that they stay
readable; everything that is skipped has to be missing from the result, the rest has
to be there."""
import numpy as np
import pytest
import torch

import fp8_ref
import paged_ref as ref
import scaled_dot_product_02_gb300 as sdpa

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
D, PAGE, HKV, PAGES = 128, 16, 2, 5
ERR_ADDRESS = 9


class Shrunk:
    """The checked library with extents 16 bytes short; .violations behind the block."""

    def __enter__(self):
        self.checked = sdpa.address_checked()
        self.checked.__enter__()
        sdpa.sdpa_debug_address_report()
        sdpa.sdpa_debug_address_shrink(16)
        return self

    def __exit__(self, *exc):
        try:
            sdpa.sdpa_debug_address_shrink(0)
            self.violations = sdpa.sdpa_debug_address_report()[0]
            error = sdpa.sdpa_get_device_error()
        finally:
            self.checked.__exit__(*exc)
        if exc[0] is None:
            assert self.violations > 0 and error == ERR_ADDRESS


def meta(room):
    """(block table, kv_lens, cu_seqlens) in the int32 tensor `room`: one sequence on the last page, all 16 of its slots."""
    tab, lens, cu = room[:4].view(1, 4), room[4:5], room[8:10]
    tab.copy_(torch.tensor([[PAGES - 1, -1, -1, -1]], dtype=torch.int32))
    lens.fill_(PAGE)
    cu.copy_(torch.tensor([0, PAGE], dtype=torch.int32))
    return tab, lens, cu


def byte(*shape, seed=0):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, 120, shape).astype(np.uint8)).cuda()


@pytest.mark.parametrize("norm", [False, True])
def test_the_append_skips_the_last_bytes(norm):
    """The last row's last 16 codes of K and V, and the last 16 scale bytes of each, keep what they held."""
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(PAGE + 2, 64 + 3 * HKV * D, generator=g).bfloat16().cuda()  # two rows behind the last sequence
    q, k, v = (wide[:, 64 + i * HKV * D:64 + (i + 1) * HKV * D].unflatten(1, (HKV, D)) for i in range(3))
    tab, lens, cu = meta(wide.view(torch.int32)[1, :32])  # in front of the second row: within k's extent, read by nobody
    caches = [byte(PAGES, PAGE, HKV, D), byte(PAGES, PAGE, HKV, D, seed=1), byte(PAGES, PAGE, HKV, seed=2), byte(PAGES, PAGE, HKV, seed=3)]
    before = [x.clone() for x in caches]
    kw = {}
    if norm:
        t = ref.angles_table(40, D).cuda()  # positions go up to 15
        w = t.view(BF)[20, :D]              # within the table's extent: all of a weight is wanted
        w.fill_(1)
        kw = dict(q=q, q_weight=w, k_weight=w, cos_sin=t)
    want = [x.clone() for x in caches]
    sdpa.sdpa_paged_append_fp8(k, v, *want, tab, lens, cu, **kw)
    assert sdpa.sdpa_get_device_error() == 0
    assert all(not torch.equal(a.flatten()[-16:], b.flatten()[-16:]) for a, b in zip(want, before))
    with Shrunk() as s:
        sdpa.sdpa_paged_append_fp8(k, v, *caches, tab, lens, cu, **kw)
    for got, full, old in zip(caches, want, before):
        got, full, old = got.flatten(), full.flatten(), old.flatten()
        assert torch.equal(got[:-16], full[:-16]) and torch.equal(got[-16:], old[-16:])
    # two vectors of codes a tensor (skipped by two lanes), a byte a row of scales
    assert s.violations >= 2 * (2 + 16)


def filled(shape, seed):
    codes, scale = fp8_ref.quantise(torch.randn(*shape, generator=torch.Generator().manual_seed(seed)), BF)
    return codes.cuda(), scale.cuda()


def read(caches, tab, lens, cu, out):
    sdpa.sdpa_paged_read_fp8(*caches, tab, lens, cu, k_out=out[0], v_out=out[1])


def values(caches):
    """The last page's rows, bf16."""
    return [fp8_ref.decode(c.cpu(), e.cpu())[-1].to(BF) for c, e in ((caches[0], caches[2]), (caches[1], caches[3]))]


def test_the_read_skips_the_last_scales_and_outputs():
    """Rows whose scale byte is outside come out as zeros, the outputs' last 16 bytes not at all."""
    (kc, ks), (vc, vs) = filled((PAGES, PAGE, HKV, D), 1), filled((PAGES, PAGE, HKV, D), 2)
    tab, lens, cu = meta(kc[0, 0].view(torch.int32).flatten())
    out = [torch.full((PAGE, HKV, D), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    with Shrunk():
        read((kc, vc, ks, vs), tab, lens, cu, out)
    for got, x in zip(out, values((kc, vc, ks, vs))):
        x[PAGE // 2:] = 0  # 16 bytes: 8 slots of 2 heads
        assert torch.equal(got.cpu().flatten()[:-8], x.flatten()[:-8])
        assert bool((got.flatten()[-8:] == 7).all())


@pytest.mark.parametrize("last", ["k", "v"])
def test_the_read_skips_the_last_codes(last):
    """Blocks of a slot: scale bytes in front, the codes of `last` at the end; those codes' last 16 come out as zeros."""
    block = torch.zeros(PAGES, PAGE, 512 + 2 * HKV * D, dtype=torch.uint8, device="cuda")
    ks, vs = block[..., :HKV], block[..., HKV:2 * HKV]
    first, second = (block[..., 512 + i * HKV * D:512 + (i + 1) * HKV * D].unflatten(-1, (HKV, D)) for i in range(2))
    kc, vc = (first, second) if last == "v" else (second, first)
    for i, (c, e) in enumerate(((kc, ks), (vc, vs))):
        codes, scale = filled((PAGES, PAGE, HKV, D), 3 + i)
        c.copy_(codes), e.copy_(scale)
    tab, lens, cu = meta(kc[0, 0].view(torch.int32).flatten() if last == "k" else block[0, 1, 16:272].view(torch.int32))
    out = [torch.full((PAGE, HKV, D), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    with Shrunk():
        read((kc, vc, ks, vs), tab, lens, cu, out)
    for name, got, x in zip("kv", out, values((kc, vc, ks, vs))):
        if name == last:
            x[-1, -1, -16:] = 0
        assert torch.equal(got.cpu().flatten()[:-8], x.flatten()[:-8])
        assert bool((got.flatten()[-8:] == 7).all())


@pytest.mark.parametrize("which", ["k", "v"])
def test_the_attention_skips_the_last_scales(which):
    """A scale byte outside counts as 127: the attention over the same codes with those bytes at 127. The other tensor's
    bytes lie within q's extent."""
    (kc, ks), (vc, vs) = filled((PAGES, PAGE, HKV, D), 5), filled((PAGES, PAGE, HKV, D), 6)
    plain = [ks.clone(), vs.clone()]
    plain[0 if which == "k" else 1][-1, PAGE // 2:] = 127
    g = torch.Generator().manual_seed(7)
    q = (torch.randn(8, 2 * HKV, D, generator=g) * 0.05).bfloat16().cuda()  # rows 2 .. 7 belong to nobody
    inside = q.view(torch.uint8)[4].flatten()[:ks.numel()].view(ks.shape)
    inside.copy_(vs if which == "k" else ks)
    ks, vs = (ks, inside) if which == "k" else (inside, vs)
    # one sequence of two tokens and 8 empty ones, whose entries are the ones outside
    tab = torch.full((9, 4), -1, dtype=torch.int32, device="cuda")
    tab[0, 0] = PAGES - 1
    lens = torch.tensor([PAGE] + [0] * 8, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + [2] * 9, dtype=torch.int32, device="cuda")
    kw = dict(max_seqlen_q=2, max_seqlen_kv=64)
    want, want_l = sdpa.sdpa_paged_fwd_fp8(q, kc, vc, *plain, tab, lens, cu, **kw)
    real, _ = sdpa.sdpa_paged_fwd_fp8(q, kc, vc, ks, vs, tab, lens, cu, **kw)
    assert not torch.equal(real[:2], want[:2])
    with Shrunk():
        got, got_l = sdpa.sdpa_paged_fwd_fp8(q, kc, vc, ks, vs, tab, lens, cu, **kw)
    assert torch.equal(got[:2], want[:2]) and torch.equal(got_l[:2], want_l[:2])


def axes_case(rows, seed):
    """(q, k, table, weight, positions): the weight lies within the table's extent, behind the positions' range."""
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(rows, h, D, generator=g).bfloat16().cuda() for h in (4, 2))
    t = ref.angles_table(300, D).cuda()
    w = t.view(BF)[90, :D]
    w.fill_(1)
    return q, k, t, w, torch.from_numpy(np.random.default_rng(seed).integers(0, 80, (3, rows)).astype(np.int32)).cuda()


SECTIONS = (16, 24, 24)


@pytest.mark.parametrize("rows", [64, 6000])
def test_the_axes_skip_the_last_positions(rows):
    """The tokens whose position on the last axis is outside are skipped whole; both kernels."""
    q, k, t, w, pos = axes_case(rows, 8)
    want = sdpa.sdpa_qk_norm_rope(q, k, w, w, t, pos, sections=SECTIONS)
    out = [torch.full_like(x, 7.0) for x in want]
    with Shrunk():
        sdpa.sdpa_qk_norm_rope(q, k, w, w, t, pos, sections=SECTIONS, q_out=out[0], k_out=out[1])
    for got, full in zip(out, want):
        assert torch.equal(got[:rows - 4], full[:rows - 4]) and bool((got[rows - 4:] == 7).all())


@pytest.mark.parametrize("rows", [64, 6000])
def test_the_axes_skip_the_last_outputs(rows):
    """Positions within the table's extent: every token is written but for the last 16 bytes of both outputs (the last
    token's inputs are short, too)."""
    q, k, t, w, pos = axes_case(rows, 8)
    want = sdpa.sdpa_qk_norm_rope(q, k, w, w, t, pos, sections=SECTIONS)
    held = t.view(torch.int32).flatten()[100 * D:100 * D + 3 * rows].view(3, rows)
    held.copy_(pos)
    out = [torch.full_like(x, 7.0) for x in want]
    with Shrunk():
        sdpa.sdpa_qk_norm_rope(q, k, w, w, t, held, sections=SECTIONS, q_out=out[0], k_out=out[1])
    for got, full in zip(out, want):
        assert torch.equal(got[:-1], full[:-1]) and bool((got.flatten()[-8:] == 7).all())


@pytest.mark.parametrize("rows", [64, 6000])
def test_the_axes_skip_the_last_angles(rows):
    """Tokens at the table's last row on the last axis: those angles are outside, the others' are not."""
    q, k, t, w, pos = axes_case(rows, 9)
    counts = []
    for last in (89, 299):
        p = pos.clone()
        p[2, 5:9] = last
        out = [torch.full((rows, h, D), 7.0, dtype=BF, device="cuda") for h in (4, 2)]
        want = sdpa.sdpa_qk_norm_rope(q, k, w, w, t, p, sections=SECTIONS)
        with Shrunk() as s:
            sdpa.sdpa_qk_norm_rope(q, k, w, w, t, p, sections=SECTIONS, q_out=out[0], k_out=out[1])
        counts.append(s.violations)
        for got, full in zip(out, want):
            keep = torch.ones(rows, dtype=torch.bool)
            keep[5:9], keep[rows - 4:] = last != 299, False
            assert torch.equal(got[keep.cuda()], full[keep.cuda()])
    assert counts[1] > counts[0]
