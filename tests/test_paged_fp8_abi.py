"""Host-side refusals of the 8-bit paged cache and of rotations with several axes (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_ref
import scaled_dot_product_02_gb300 as sdpa
from test_paged_abi import BASE, M, PTR, built, norm_problem, paged_problem  # noqa: F401 (built: the module's fixture)


def axes(*pairs, n=None, stride=0):
    a = sdpa.RopeAxes()
    a.num_axes = len(pairs) if n is None else n
    for i, x in enumerate(pairs):
        a.pairs[i] = x
    a.position_stride = stride
    return a


def scales(**kw):
    s = sdpa.PagedScales()
    base = dict(k=BASE + 40 * M, v=BASE + 41 * M, k_page_stride=32, k_slot_stride=2, k_head_stride=1, v_page_stride=32,
                v_slot_stride=2, v_head_stride=1)
    base.update(kw)
    for k, v in base.items():
        setattr(s, k, v)
    return s


def ref(x):
    return None if x is None else ctypes.byref(x)


def ptrs(a):
    return [PTR(x) if x else None for x in a.values()]


def test_axes_refusals():
    def call(p, a, **kw):
        x = dict(q=BASE, k=BASE + M, wq=BASE + 2 * M, wk=BASE + 3 * M, t=BASE + 4 * M, pos=BASE + 5 * M, qo=BASE + 6 * M,
                 ko=BASE + 7 * M)
        x.update(kw)
        return sdpa.lib().sdpa_qk_norm_rope_axes(ref(p), ref(a), *ptrs(x), None)

    ok = norm_problem()
    assert call(norm_problem(rows=0), axes(16, 24, 24)) == 0
    assert call(ok, None) == 1 and call(None, axes(64)) == 1
    for bad in (axes(16, 24, 25), axes(16, 24, 23), axes(64, 0), axes(0, 64), axes(-1, 65), axes(64, n=0), axes(13, 13, 13, 25, n=5),
                axes(2 ** 31 - 1, 65), axes(16, 24, 24, stride=99), axes(64, stride=-100), axes(64, stride=1 << 36)):
        assert call(norm_problem(rows=100), bad) == 1, list(bad.pairs)
        assert call(norm_problem(rows=100), bad, q=None) == 1
    assert call(norm_problem(rotary_dim=0), axes(1, n=1)) == 1
    for name in ("q", "k", "wq", "wk", "qo", "ko", "t", "pos"):
        assert call(ok, axes(16, 24, 24), **{name: None}) == 1, name
    # the positions' extent is every axis's
    assert call(ok, axes(16, 24, 24), qo=BASE + 5 * M + 2 * 400) == 4
    assert call(ok, axes(16, 48, stride=M // 4), qo=BASE + 6 * M) == 4

    def back(p, a, **kw):
        x = dict(gq=BASE, gk=BASE + M, q=BASE + 2 * M, k=BASE + 3 * M, wq=BASE + 4 * M, wk=BASE + 5 * M, t=BASE + 6 * M,
                 pos=BASE + 7 * M, dq=BASE + 8 * M, dk=BASE + 9 * M, dwq=BASE + 10 * M, dwk=BASE + 11 * M)
        x.update(kw)
        n = sdpa.lib().sdpa_qk_norm_rope_bwd_workspace_size(ref(p))
        return sdpa.lib().sdpa_qk_norm_rope_axes_bwd(ref(p), ref(a), *ptrs(x), PTR(BASE + 20 * M), n, None)

    assert back(ok, None) == 1 and back(ok, axes(16, 24, 25)) == 1 and back(ok, axes(64), dq=BASE + 2 * M) == 4
    assert back(ok, axes(16, 24, 24), dk=BASE + 7 * M + 800) == 4


def append(p, n=None, a=None, s=None, **kw):
    x = dict(q=BASE, k=BASE + M, v=BASE + 2 * M, wq=BASE + 3 * M, wk=BASE + 4 * M, t=BASE + 5 * M, pos=BASE + 6 * M,
             qo=BASE + 7 * M, kc=BASE + 8 * M, vc=BASE + 20 * M, cu=BASE + 30 * M, lens=BASE + 31 * M, tab=BASE + 32 * M)
    x.update(kw)
    return sdpa.lib().sdpa_paged_append_fp8(ref(p), ref(n), ref(a), ref(s), *ptrs(x), None)


def test_append_refusals():
    ok, n = paged_problem(), norm_problem()
    assert append(ok, s=None) == 1 and append(None, s=scales()) == 1
    assert append(paged_problem(total_q=0), s=scales()) == 0
    for bad in (dict(k=None), dict(v=None), dict(k_page_stride=0), dict(k_slot_stride=-1), dict(v_head_stride=0),
                dict(v_page_stride=1 << 36)):
        assert append(ok, s=scales(**bad)) == 1, bad
    # codes move 16 bytes at a time
    d = dict(k_slot_stride=264, k_page_stride=16 * 264, k_head_stride=132)
    assert append(paged_problem(**d), s=scales()) == 1
    d = dict(k_slot_stride=272, k_page_stride=16 * 272, k_head_stride=136, v_slot_stride=272, v_page_stride=16 * 272, v_head_stride=136)
    assert append(paged_problem(**d), s=scales()) == 1
    # a page with room for scale bytes only behind its codes: no stride of a copy
    d = {x + "_page_stride": 16 * 2 * 128 + 32 for x in "kv"}
    assert append(paged_problem(**d), s=scales()) == 2
    for name in ("k", "v", "kc", "vc", "cu", "lens", "tab"):
        assert append(ok, s=scales(), **{name: None}) == 1, name
    for name in ("k", "v", "kc", "vc"):
        at = {"k": 1, "v": 2, "kc": 8, "vc": 20}[name]
        assert append(ok, s=scales(), **{name: BASE + at * M + 8}) == 3, name
    for name in ("q", "wq", "wk", "qo", "t"):
        assert append(ok, n, s=scales(), **{name: None}) == 1, name
    # several axes: with a norm and rotation, and with positions
    assert append(ok, None, axes(64), scales()) == 1
    assert append(ok, n, axes(16, 24, 24), scales(), pos=None) == 1
    assert append(ok, n, axes(16, 24, 25), scales()) == 1
    # nothing may be written over an input or another output
    codes = 300 * 16 * 2 * 128
    assert append(ok, s=scales(k=BASE + M)) == 4                      # scale bytes over k
    assert append(ok, s=scales(v=BASE + 8 * M + codes - 1)) == 4      # over the last code
    assert append(ok, s=scales(v=BASE + 40 * M)) == 4                 # over the other scales
    assert append(ok, s=scales(k_slot_stride=1)) == 4                 # a row's byte over another's
    assert append(ok, s=scales(k_page_stride=16)) == 4                # a page's over the next one's
    assert append(ok, n, s=scales(k=BASE + 7 * M)) == 4               # over q_out
    assert append(ok, s=scales(), vc=BASE + 8 * M + 128) == 4
    assert append(ok, s=scales(), cu=BASE + 40 * M + 300 * 32 - 4) == 4


def test_append_axes_refusals():
    def call(p, n, a, **kw):
        x = dict(q=BASE, k=BASE + M, v=BASE + 2 * M, wq=BASE + 3 * M, wk=BASE + 4 * M, t=BASE + 5 * M, pos=BASE + 6 * M,
                 qo=BASE + 7 * M, kc=BASE + 8 * M, vc=BASE + 20 * M, cu=BASE + 30 * M, lens=BASE + 31 * M, tab=BASE + 32 * M)
        x.update(kw)
        return sdpa.lib().sdpa_paged_append_axes(ref(p), ref(n), ref(a), *ptrs(x), None)

    ok, n = paged_problem(), norm_problem()
    assert call(ok, n, None) == 1 and call(ok, None, axes(64)) == 1 and call(ok, n, axes(64), pos=None) == 1
    assert call(ok, n, axes(63)) == 1 and call(ok, n, axes(32, 32, stride=39)) == 1
    assert call(paged_problem(total_q=0), n, axes(32, 32)) == 0


def test_read_refusals():
    def call(p, s, **kw):
        x = dict(kc=BASE + 8 * M, vc=BASE + 20 * M, ko=BASE, vo=BASE + M, cu=BASE + 30 * M, lens=BASE + 31 * M, tab=BASE + 32 * M)
        x.update(kw)
        return sdpa.lib().sdpa_paged_read_fp8(ref(p), ref(s), *ptrs(x), None)

    ok = paged_problem()
    assert call(None, scales()) == 1 and call(ok, None) == 1 and call(ok, scales(v=None)) == 1
    assert call(paged_problem(total_q=0), scales()) == 0 and call(paged_problem(batch=0), scales()) == 0
    for name in ("kc", "vc", "ko", "vo", "cu", "lens", "tab"):
        assert call(ok, scales(), **{name: None}) == 1, name
    for name, at in (("kc", 8), ("vc", 20), ("ko", 0), ("vo", 1)):
        assert call(ok, scales(), **{name: BASE + at * M + 4}) == 3, name
    assert call(ok, scales(), vo=BASE + 40 * 256 * 2 - 16) == 4          # over the last row of k_out
    assert call(ok, scales(), ko=BASE + 8 * M) == 4 and call(ok, scales(), vo=BASE + 40 * M) == 4
    wide = paged_problem(k_stride=512, v_stride=512)                     # slices of one tensor's rows
    assert call(wide, scales(), vo=BASE + 256 * 2 - 16) == 4
    assert call(paged_problem(k_stride=512, v_stride=520), scales(), vo=BASE + 512) == 4


def test_attention_refusals():
    def call(p, s, ws=BASE + 50 * M, n=None, **kw):
        x = dict(q=BASE, kc=BASE + 8 * M, vc=BASE + 20 * M, o=BASE + M, lse=BASE + 2 * M, cu=BASE + 30 * M, lens=BASE + 31 * M,
                 tab=BASE + 32 * M)
        x.update(kw)
        n = sdpa.lib().sdpa_paged_fwd_fp8_workspace_size(ref(p)) if n is None else n
        return sdpa.lib().sdpa_paged_fwd_fp8(ref(p), ref(s), *ptrs(x), PTR(ws) if ws else None, n, None)

    ok = paged_problem()
    need = sdpa.lib().sdpa_paged_fwd_fp8_workspace_size(ref(ok))
    assert 0 < need <= sdpa.PAGED_WORKSPACE_MAX
    assert call(None, scales()) == 1 and call(ok, None) == 1 and call(ok, scales(k=None)) == 1
    assert call(paged_problem(head_dim=64), scales()) == 2 and call(paged_problem(mask_type=1), scales()) == 2
    assert call(paged_problem(total_q=0), scales()) == 0
    assert call(ok, scales(), n=need - 1) == 5 and call(ok, scales(), ws=None) == 5 and call(ok, scales(), ws=BASE + 50 * M + 128) == 3
    for name in ("q", "kc", "vc", "o", "lse", "cu", "lens", "tab"):
        assert call(ok, scales(), **{name: None}) == 1, name
    for name, at in (("q", 0), ("kc", 8), ("vc", 20), ("o", 1), ("lse", 2)):
        assert call(ok, scales(), **{name: BASE + at * M + 4}) == 3, name
    assert call(ok, scales(), o=BASE) == 4 and call(ok, scales(), lse=BASE + 40 * M) == 4
    assert call(ok, scales(), ws=BASE + 41 * M - 256) == 4 and call(ok, scales(), o=BASE + 2 * M) == 4
    for d, dv in ((128, 0), (192, 128), (256, 0), (512, 0)):
        for hq, hkv in ((8, 2), (128, 1), (65536, 65536)):
            for batch, q, kv in ((1, 1, 1 << 30), (1 << 20, 1, 4096), (1, 1 << 20, 1 << 20), (500, 64, 1 << 20)):
                p = paged_problem(head_dim=d, head_dim_v=dv, num_heads_q=hq, num_heads_kv=hkv, batch=batch, seqlen_q=q,
                                  total_q=batch * q, seqlen_kv=kv, page_size=1 << 16, max_pages=1 << 14)
                assert sdpa.lib().sdpa_paged_fwd_fp8_workspace_size(ref(p)) <= sdpa.PAGED_WORKSPACE_MAX


# ---------------------------------------------------------------- the binding

def tensors(order="nhd", d=128, dv=128, hkv=2, pages=9, page=16):
    heads = (pages, page, hkv) if order == "nhd" else (pages, hkv, page)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return dict(kc=u8(*heads, d), vc=u8(*heads, dv), ks=u8(*heads), vs=u8(*heads), tab=torch.zeros(3, 4, dtype=torch.int32),
                lens=i32(5, 6, 7), cu=i32(0, 1, 2, 4))


CACHE = ("kc", "vc", "ks", "vs", "tab", "lens", "cu")


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(sdpa, "_refuse_cpu", lambda t: None)
    monkeypatch.setattr(sdpa, "_launch", lambda name, device, *args: seen.append((name, args)))
    return seen


def test_binding_marshals(calls):
    x = torch.zeros(4, 6 * 128, dtype=torch.bfloat16)
    q, k, v = (x[:, a:b].unflatten(1, (-1, 128)) for a, b in ((0, 256), (256, 512), (512, 768)))
    w = torch.ones(128, dtype=torch.bfloat16)
    cs, pos = torch.zeros(50, 128), torch.zeros(3, 9, dtype=torch.int32)[:, 2:6]
    for order in ("nhd", "hnd"):
        t = tensors(order)
        out = sdpa.sdpa_paged_append_fp8(k, v, *(t[n] for n in CACHE), cache_layout=order, q=q, q_weight=w, k_weight=w, cos_sin=cs,
                                         positions=pos, sections=[16, 24, 24])
        assert out.shape == q.shape and out.is_contiguous()
        name, args = calls.pop()
        p, n, a, s = (y._obj for y in args[:4])
        assert name == "sdpa_paged_append_fp8" and n.rotary_dim == 128 and p.k_stride == 768
        assert (a.num_axes, list(a.pairs), a.position_stride) == (3, [16, 24, 24, 0], 9)
        assert (s.k_page_stride, s.k_slot_stride, s.k_head_stride) == ((32, 2, 1) if order == "nhd" else (32, 1, 16))
        assert s.k == t["ks"].data_ptr() and s.v == t["vs"].data_ptr()
        sdpa.sdpa_paged_append_fp8(k, v, *(t[n] for n in CACHE), cache_layout=order)
        assert calls.pop()[1][1:3] == (None, None)
        ko, vo = sdpa.sdpa_paged_read_fp8(*(t[n] for n in CACHE), cache_layout=order, rows=11, dtype=torch.float16)
        assert ko.shape == vo.shape == (11, 2, 128) and ko.dtype is torch.float16
        name, args = calls.pop()
        assert name == "sdpa_paged_read_fp8" and args[0]._obj.total_q == 11 and args[0]._obj.dtype == 1
        o, lse = sdpa.sdpa_paged_fwd_fp8(q, *(t[n] for n in CACHE), cache_layout=order, max_seqlen_q=2)
        assert o.shape == (4, 2, 128) and lse.shape == (4, 2)
        assert calls.pop()[0] == "sdpa_paged_fwd_fp8"
    # one sequence of one page with one head: strides of single entries are free
    t = tensors(hkv=1, pages=1)
    for n in ("ks", "vs"):
        t[n] = t[n].as_strided(t[n].shape, (0, 1, 0))
    sdpa.sdpa_paged_fwd_fp8(q, *(t[n] for n in CACHE), max_seqlen_q=2)
    s = calls.pop()[1][1]._obj
    assert min(s.k_page_stride, s.k_slot_stride, s.k_head_stride) >= 1
    sdpa.sdpa_qk_norm_rope(q, k, w, w, cs, pos, sections=(16, 24, 24))
    sdpa.sdpa_qk_norm_rope(q, k, w, w, cs, pos[0])
    assert [c[0] for c in calls] == ["sdpa_qk_norm_rope_axes", "sdpa_qk_norm_rope"]


def test_binding_refusals(calls):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    cs, pos = torch.zeros(50, 128), torch.zeros(3, 4, dtype=torch.int32)
    for change in (dict(kc=torch.bfloat16), dict(ks=torch.int8), dict(vs=(9, 16, 3)), dict(ks=(9, 2, 16)), dict(vc=(9, 16, 3, 128)),
                   dict(lens=(4,)), dict(cu=(3,)), dict(vs="broadcast"), dict(tab=torch.int64)):
        t = tensors()
        for n, c in change.items():
            t[n] = (t[n].to(c) if isinstance(c, torch.dtype) else t[n][:, :, :1].expand(-1, -1, 2) if c == "broadcast"
                    else torch.zeros(c, dtype=t[n].dtype))
        if change.get("kc") is torch.bfloat16:
            t["vc"] = t["vc"].to(torch.bfloat16)
        with pytest.raises(ValueError):
            sdpa.sdpa_paged_append_fp8(x, x, *(t[n] for n in CACHE))
        with pytest.raises(ValueError):
            sdpa.sdpa_paged_fwd_fp8(x, *(t[n] for n in CACHE), max_seqlen_q=2)
        with pytest.raises(ValueError):
            sdpa.sdpa_paged_read_fp8(*(t[n] for n in CACHE), rows=4, dtype=torch.bfloat16)
    t = tensors()
    cache = [t[n] for n in CACHE]
    for kw in (dict(), dict(rows=4), dict(dtype=torch.bfloat16), dict(rows=4, dtype=torch.float32), dict(rows=5, k_out=x),
               dict(k_out=x, v_out=x[:3]), dict(k_out=x, v_out=x.half()), dict(k_out=x[:, :1]), dict(k_out=x[..., :64])):
        with pytest.raises(ValueError):
            sdpa.sdpa_paged_read_fp8(*cache, **kw)
    for kw in (dict(sections=(16, 24)), dict(sections=(64, 0)), dict(sections=(16, 24, 25)), dict(sections=()),
               dict(sections=(16, 16, 16, 8, 8)), dict(sections=(16, 24, 24), positions=None),
               dict(sections=(16, 24, 24), positions=pos[:2]), dict(sections=(16, 24, 24), positions=pos[:, :3]),
               dict(sections=(16, 24, 24), positions=pos[:1].expand(3, -1)), dict(sections=(16, 24, 24), positions=pos.long()),
               dict(sections=(16, 24, 24), positions=torch.zeros(4, 3, dtype=torch.int32).T), dict(sections=(64,), cos_sin=None)):
        kw = {"cos_sin": cs, "positions": pos, **kw}
        with pytest.raises(ValueError):
            sdpa.sdpa_qk_norm_rope(x, x, w, w, **kw)
        with pytest.raises(ValueError):
            sdpa.sdpa_qk_norm_rope_bwd(x, x, x, x, w, w, **kw)
        with pytest.raises(ValueError):
            sdpa.sdpa_paged_append_fp8(x, x, *cache, q=x, q_weight=w, k_weight=w, **kw)
    with pytest.raises(ValueError):
        sdpa.sdpa_paged_append_fp8(x, x, *cache, sections=(64,))
    assert not calls


def test_reference_quantiser():
    """The tests' own quantiser against torch's conversion, and its exponents against their definition."""
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(300, 64, generator=g) * torch.exp2(torch.randn(300, 1, generator=g) * 6)).bfloat16()
    codes, scale = fp8_ref.quantise(x, torch.bfloat16)
    y = torch.ldexp(x.float(), 127 - scale.int()[:, None])
    assert bool((y.abs().amax(1) <= 448).all()) and bool((y.abs().amax(1) > 224).all())
    assert torch.equal(codes, y.to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.equal(fp8_ref.decode(codes, scale), torch.ldexp(codes.view(torch.float8_e4m3fn).float(), scale.int()[:, None] - 127).double())
    assert np.array_equal(fp8_ref.exponent(np.array([0, 448, 448.1, 2.0 ** -200, 2.0 ** 200, np.inf]), torch.bfloat16),
                          [-80, 0, 1, -80, 80, 80])
    # every code is exact in the 16-bit types at the ends of their exponents
    v = torch.from_numpy(fp8_ref.VALUES[~np.isnan(fp8_ref.VALUES)])
    for dtype, ends in fp8_ref.LIMITS.items():
        for e in ends:
            assert torch.equal((v * 2.0 ** e).to(dtype).double(), v * 2.0 ** e)
