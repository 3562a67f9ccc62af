"""Host-side refusals of the norm + rotation and paged-cache entry points (no GPU)."""
import ctypes

import pytest
import torch

import scaled_dot_product_02_gb300 as sdpa

PTR = ctypes.c_void_p
BASE = 1 << 40
M = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def built():
    from scaled_dot_product_02_gb300 import build

    build.build()


def norm_problem(**kw):
    p = sdpa.NormRopeProblem()
    base = dict(dtype=0, num_heads_q=8, num_heads_kv=2, head_dim=128, rotary_dim=128, interleaved=0, eps=1e-6,
                max_positions=1000, rows=100, q_stride=0, k_stride=0, dq_stride=0, dk_stride=0)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


def paged_problem(**kw):
    p = sdpa.PagedProblem()
    base = dict(dtype=0, batch=4, num_heads_q=8, num_heads_kv=2, head_dim=128, head_dim_v=0, total_q=40, seqlen_q=10,
                seqlen_kv=1000, page_size=16, num_pages=300, max_pages=63, mask_type=2, window_left=-1,
                softmax_scale=0.1, table_stride=0, q_stride=0, k_stride=0, v_stride=0)
    d = kw.get("head_dim", 128)
    base.update(k_page_stride=16 * 2 * d, k_slot_stride=2 * d, k_head_stride=d, v_page_stride=16 * 2 * d,
                v_slot_stride=2 * d, v_head_stride=d)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


def norm_call(p, **kw):
    a = dict(q=BASE, k=BASE + M, wq=BASE + 2 * M, wk=BASE + 3 * M, t=BASE + 4 * M, pos=BASE + 5 * M, qo=BASE + 6 * M,
             ko=BASE + 7 * M)
    a.update(kw)
    return sdpa.lib().sdpa_qk_norm_rope(ctypes.byref(p) if p is not None else None, *[PTR(x) if x else None for x in a.values()],
                                        None)


def test_norm_rope_refusals():
    assert norm_call(None) == 1
    assert norm_call(norm_problem(rows=0)) == 0
    for bad, code in ((dict(dtype=2), 2), (dict(head_dim=64), 2), (dict(num_heads_q=0), 1), (dict(num_heads_kv=-1), 1),
                      (dict(rows=-1), 1), (dict(rotary_dim=8), 1), (dict(rotary_dim=144), 1), (dict(rotary_dim=-16), 1),
                      (dict(max_positions=0), 1), (dict(interleaved=2), 1), (dict(eps=-1.0), 1),
                      (dict(eps=float("nan")), 1), (dict(q_stride=1000), 1), (dict(q_stride=1028), 1),
                      (dict(rows=1 << 31), 2)):
        assert norm_call(norm_problem(**bad)) == code, bad
    ok = norm_problem()
    for name in ("q", "k", "wq", "wk", "qo", "ko", "t", "pos"):
        assert norm_call(ok, **{name: None}) == 1, name
    for name in ("q", "k", "wq", "wk", "qo", "ko", "t"):
        at = {"q": 0, "k": 1, "wq": 2, "wk": 3, "t": 4, "qo": 6, "ko": 7}[name]
        assert norm_call(ok, **{name: BASE + at * M + 8}) == 3, name
    assert norm_call(ok, qo=BASE + 64) == 4           # in place is refused too
    assert norm_call(ok, ko=BASE + 6 * M + 100 * 8 * 128 * 2 - 16) == 4
    # a row further down a strided q is part of its extent
    assert norm_call(norm_problem(q_stride=4096), ko=BASE + 99 * 4096 * 2) == 4


def test_norm_rope_bwd_refusals():
    def call(p, ws=BASE + 20 * M, n=None, **kw):
        a = dict(gq=BASE, gk=BASE + M, q=BASE + 2 * M, k=BASE + 3 * M, wq=BASE + 4 * M, wk=BASE + 5 * M, t=BASE + 6 * M,
                 pos=BASE + 7 * M, dq=BASE + 8 * M, dk=BASE + 9 * M, dwq=BASE + 10 * M, dwk=BASE + 11 * M)
        a.update(kw)
        n = sdpa.lib().sdpa_qk_norm_rope_bwd_workspace_size(ctypes.byref(p)) if n is None else n
        return sdpa.lib().sdpa_qk_norm_rope_bwd(ctypes.byref(p), *[PTR(x) if x else None for x in a.values()],
                                                PTR(ws) if ws else None, n, None)

    ok = norm_problem()
    assert sdpa.lib().sdpa_qk_norm_rope_bwd_workspace_size(ctypes.byref(norm_problem(head_dim=64))) == 0
    assert call(ok, n=16) == 5 and call(ok, ws=None) == 5 and call(ok, ws=BASE + 20 * M + 8) == 3
    for name in ("gq", "gk", "q", "k", "wq", "wk", "t", "pos", "dq", "dk", "dwq", "dwk"):
        assert call(ok, **{name: None}) == 1, name
    assert call(ok, dq=BASE + 2 * M) == 4             # dq over q
    assert call(ok, dwq=BASE + 20 * M) == 4           # dw over the workspace
    assert call(ok, dk=BASE + 8 * M + 1024) == 4      # dk inside dq
    # slices of one fused gradient interleave, but may not share values
    w = (8 + 2 + 2) * 128
    fused = norm_problem(dq_stride=w, dk_stride=w)
    assert call(fused, dk=BASE + 8 * M + (8 * 128 - 8) * 2) == 4
    assert call(norm_problem(dq_stride=w, dk_stride=w + 8), dk=BASE + 8 * M + 8 * 128 * 2) == 4


def test_paged_refusals():
    check = lambda **kw: sdpa.sdpa_check_paged(paged_problem(**kw))  # noqa: E731
    assert check() == 0 and check(head_dim=192, head_dim_v=128) == 0 and check(head_dim=192) == 0
    assert check(head_dim=512) == 0 and check(mask_type=0) == 0 and check(window_left=0) == 0
    for bad, code in ((dict(dtype=3), 2), (dict(head_dim=64), 2), (dict(head_dim=128, head_dim_v=64), 2),
                      (dict(head_dim_v=-1), 1), (dict(batch=-1), 1), (dict(total_q=-1), 1), (dict(seqlen_kv=-1), 1),
                      (dict(num_heads_q=7), 1), (dict(page_size=0), 1), (dict(page_size=24), 2), (dict(num_pages=0), 1),
                      (dict(max_pages=62), 1), (dict(table_stride=10), 1), (dict(mask_type=1), 2), (dict(mask_type=3), 1),
                      (dict(window_left=-2), 1), (dict(mask_type=0, window_left=5), 2), (dict(softmax_scale=-1.0), 1),
                      (dict(softmax_scale=float("inf")), 1), (dict(k_slot_stride=100), 1), (dict(v_head_stride=132), 1),
                      (dict(k_page_stride=0), 1), (dict(q_stride=512), 1),
                      (dict(seqlen_kv=(1 << 30) + 1, max_pages=1 << 27), 2), (dict(batch=(1 << 20) + 1), 2), (dict(k_stride=260), 1)):
        assert check(**bad) == code, bad


def test_append_refusals():
    def call(p, n=None, **kw):
        a = dict(q=BASE, k=BASE + M, v=BASE + 2 * M, wq=BASE + 3 * M, wk=BASE + 4 * M, t=BASE + 5 * M, pos=BASE + 6 * M,
                 qo=BASE + 7 * M, kc=BASE + 8 * M, vc=BASE + 20 * M, cu=BASE + 30 * M, lens=BASE + 31 * M, tab=BASE + 32 * M)
        a.update(kw)
        return sdpa.lib().sdpa_paged_append(ctypes.byref(p), ctypes.byref(n) if n is not None else None,
                                            *[PTR(x) if x else None for x in a.values()], None)

    ok = paged_problem()
    assert call(paged_problem(total_q=0)) == 0 and call(paged_problem(batch=0)) == 0
    assert call(paged_problem(page_size=8)) == 2
    for name in ("k", "v", "kc", "vc", "cu", "lens", "tab"):
        assert call(ok, **{name: None}) == 1, name
    assert call(ok, k=BASE + M + 2) == 3 and call(ok, vc=BASE + 20 * M + 8) == 3
    assert call(ok, k=BASE + 8 * M + 4096) == 4       # new rows inside the cache
    assert call(ok, tab=BASE + 20 * M) == 4           # the block table inside the cache
    n = norm_problem(rotary_dim=24)
    assert call(ok, n) == 1
    n = norm_problem()
    for name in ("q", "wq", "wk", "t", "qo"):
        assert call(ok, n, **{name: None}) == 1, name
    assert call(ok, n, qo=BASE + 64) == 4 and call(ok, n, qo=BASE + 8 * M) == 4


def test_paged_fwd_refusals():
    def call(p, n=None, **kw):
        a = dict(q=BASE, kc=BASE + M, vc=BASE + 12 * M, o=BASE + 24 * M, lse=BASE + 25 * M, cu=BASE + 26 * M,
                 lens=BASE + 27 * M, tab=BASE + 28 * M, ws=BASE + 30 * M)
        a.update(kw)
        n = sdpa.sdpa_paged_fwd_workspace_size(p) if n is None else n
        return sdpa.lib().sdpa_paged_fwd(ctypes.byref(p), *[PTR(x) if x else None for x in a.values()], n, None)

    ok = paged_problem()
    assert call(paged_problem(total_q=0)) == 0 and call(paged_problem(batch=0)) == 0
    assert call(paged_problem(head_dim=64)) == 2 and call(paged_problem(mask_type=1)) == 2
    for name in ("q", "kc", "vc", "o", "lse", "cu", "lens", "tab"):
        assert call(ok, **{name: None}) == 1, name
    for name, at in (("q", 0), ("kc", 1), ("vc", 12), ("o", 24), ("lse", 25)):
        assert call(ok, **{name: BASE + at * M + 8}) == 3, name
    assert call(ok, n=0) == 5 and call(ok, ws=None) == 5 and call(ok, ws=BASE + 30 * M + 16) == 3
    assert call(ok, n=sdpa.sdpa_paged_fwd_workspace_size(ok) - 1) == 5
    assert call(ok, o=BASE + M + 4096) == 4 and call(ok, lse=BASE + 24 * M) == 4 and call(ok, o=BASE + 30 * M) == 4
    assert call(ok, tab=BASE + 30 * M + 256) == 4
    assert call(paged_problem(q_stride=8 * 128 + 8)) == 2
    # cache strides that are not multiples of one another, or K and V in different orders
    assert sdpa.sdpa_check_paged(paged_problem(k_page_stride=16 * 256 + 8)) == 2
    assert sdpa.sdpa_check_paged(paged_problem(k_slot_stride=264)) == 2
    assert sdpa.sdpa_check_paged(paged_problem(v_slot_stride=128, v_head_stride=2048)) == 2
    assert sdpa.sdpa_check_paged(paged_problem(num_heads_kv=1, k_head_stride=8 * 99, v_head_stride=4096)) == 0


@pytest.mark.parametrize("d,dv", [(128, 128), (192, 128), (256, 256), (512, 512)])
def test_the_paged_workspace_is_bounded(d, dv):
    most = 0
    for hq, hkv in ((1, 1), (8, 2), (32, 8), (128, 1), (300, 1)):
        for batch, new, kv in ((1, 1, 1), (1, 1, 1 << 20), (64, 1, 16384), (4096, 8, 1 << 17), (3, 5000, 1 << 17)):
            p = paged_problem(num_heads_q=hq, num_heads_kv=hkv, head_dim=d, head_dim_v=dv, batch=batch, total_q=batch * new,
                              seqlen_q=new, seqlen_kv=kv, max_pages=kv // 16 + 1, k_page_stride=16 * hkv * d,
                              k_slot_stride=hkv * d, k_head_stride=d, v_page_stride=16 * hkv * dv, v_slot_stride=hkv * dv,
                              v_head_stride=dv)
            assert sdpa.sdpa_check_paged(p) == 0
            n = sdpa.sdpa_paged_fwd_workspace_size(p)
            assert n > 0
            most = max(most, n)
    assert most <= sdpa.PAGED_WORKSPACE_MAX


def test_binding_refuses_what_does_not_fit():
    bf = torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731
    q, k, w = z(6, 4, 128), z(6, 2, 128), z(128)
    pos, table = z(6, dt=torch.int32), torch.zeros(50, 128)
    f = sdpa.sdpa_qk_norm_rope
    with pytest.raises(ValueError, match="CUDA"):
        f(q, k, w, w, table, pos)
    for args in ((q, z(5, 2, 128), w, w, table, pos), (q, z(6, 2, 256), w, w, table, pos), (q, k, z(64), w, table, pos),
                 (q, k, w, w.float(), table, pos), (q, k, w, w, table.half(), pos), (q, k, w, w, table, pos.long()),
                 (q, k, w, w, table, pos[:5]), (q, k, w, w, table, None), (q, k.half(), w, w, table, pos),
                 (q.float(), k.float(), w.float(), w.float(), table, pos), (q.transpose(1, 2), k, w, w, table, pos),
                 (z(4, 6, 128).transpose(0, 1), k, w, w, table, pos)):
        with pytest.raises(ValueError):
            f(*args)
    kc, vc = z(9, 16, 2, 128), z(9, 16, 2, 128)
    tab, lens, cu = z(2, 4, dt=torch.int32), z(2, dt=torch.int32), z(3, dt=torch.int32)
    a = sdpa.sdpa_paged_append
    good = dict(k=k, v=k, k_cache=kc, v_cache=vc, block_table=tab, kv_lens=lens, cu_seqlens_q=cu)
    with pytest.raises(ValueError, match="CUDA"):
        a(**good)
    for bad in (dict(k=z(6, 3, 128)), dict(v=z(5, 2, 128)), dict(k_cache=z(9, 2, 16, 128)), dict(v_cache=z(9, 16, 2, 256)),
                dict(block_table=tab.long()), dict(kv_lens=lens[:1]), dict(cu_seqlens_q=cu[:2]), dict(cache_layout="dnh"),
                dict(q=z(6, 4, 128)), dict(q=z(5, 4, 128), q_weight=w, k_weight=w), dict(cos_sin=table),
                dict(k_cache=kc.half()), dict(q=q, q_weight=w, k_weight=w, cos_sin=table[:, :64].t())):
        with pytest.raises(ValueError):
            a(**{**good, **bad})


    a = sdpa.sdpa_paged_fwd
    good = dict(q=q, k_cache=kc, v_cache=vc, block_table=tab, kv_lens=lens, cu_seqlens_q=cu, max_seqlen_q=6)
    with pytest.raises(ValueError, match="CUDA"):
        a(**good)
    for bad in (dict(q=z(6, 4, 256)), dict(q=z(6, 5, 128)), dict(q=z(1, 6, 4, 128)), dict(window=(4, 3)),
                dict(kv_lens=lens.long()), dict(k_cache=kc[:5]), dict(block_table=tab[:, ::2]), dict(cache_layout="hnd")):
        with pytest.raises(ValueError):
            a(**{**good, **bad})
    with pytest.raises(KeyError):
        a(**{**good, "mask": "causal_tl"})


def test_new_error_has_a_string():
    assert "table" in sdpa.error_string(10)


# ---- calls from Python

def _batch(tokens=6, batch=3, dtype=torch.bfloat16):
    return dict(q=torch.zeros(tokens, 4, 128, dtype=dtype), k=torch.zeros(tokens, 2, 128, dtype=dtype),
                v=torch.zeros(tokens, 2, 128, dtype=dtype), kc=torch.zeros(8, 16, 2, 128, dtype=dtype),
                vc=torch.zeros(8, 16, 2, 128, dtype=dtype), table=torch.zeros(batch, 4, dtype=torch.int32),
                lens=torch.full((batch,), 2, dtype=torch.int32),
                cu=torch.arange(batch + 1, dtype=torch.int32) * (tokens // batch), w=torch.ones(128, dtype=dtype))


def _paged(c, **kw):
    return sdpa.sdpa_paged_fwd(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], **{"max_seqlen_q": 2, **kw})


@pytest.mark.parametrize("lead", [(6,), (2, 3), (1, 6)])
@pytest.mark.parametrize("dim", [0, -1])
def test_broadcast_tokens_are_refused(lead, dim):
    """A stride of zero in C stands for contiguous rows: an expanded tensor holds fewer rows than that."""
    one = list(lead)
    one[dim if dim == 0 and lead[0] > 1 else -1] = 1
    wide, w = torch.zeros(*lead, 4, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    thin = torch.zeros(*one, 4, 128, dtype=torch.bfloat16).expand(*lead, 4, 128)
    for q, k in ((thin, wide), (wide, thin)):
        with pytest.raises(ValueError, match="evenly spaced rows"):
            sdpa.sdpa_qk_norm_rope(q, k, w, w)
        with pytest.raises(ValueError, match="evenly spaced rows"):
            sdpa.sdpa_qk_norm_rope_bwd(wide, wide, q, k, w, w)
    with pytest.raises(ValueError, match="evenly spaced rows"):
        sdpa.sdpa_qk_norm_rope_bwd(wide, wide, wide, wide, w, w, dq=thin)


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_broadcast_tokens_of_a_batch_are_refused(name):
    c = _batch()
    c[name] = c[name][:1].expand(6, -1, -1)
    with pytest.raises(ValueError, match="evenly spaced rows"):
        if name == "q":
            _paged(c)
        sdpa.sdpa_paged_append(c["k"], c["v"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"])


@pytest.mark.parametrize("shape", ["expanded", "overlapping"])
def test_a_block_table_whose_rows_overlap_is_refused(shape):
    c = _batch()
    c["table"] = (torch.zeros(1, 4, dtype=torch.int32).expand(3, 4) if shape == "expanded"
                  else torch.zeros(8, dtype=torch.int32).as_strided((3, 4), (2, 1)))
    with pytest.raises(ValueError, match="block_table"):
        _paged(c)
    with pytest.raises(ValueError, match="block_table"):
        sdpa.sdpa_paged_append(c["k"], c["v"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"])

def test_scalars_given_as_tensors_are_read_on_every_call(monkeypatch):
    seen = []
    monkeypatch.setattr(sdpa, "_refuse_cpu", lambda t: None)
    monkeypatch.setattr(sdpa, "_launch", lambda name, device, *args: seen.append(
        next(a._obj for a in args if hasattr(a, "_obj"))))
    c = _batch()
    most, scale, left = torch.tensor(2), torch.tensor(0.5), torch.tensor(4)
    for n in (2, 5):
        most.fill_(n), scale.fill_(n / 4), left.fill_(n + 8)
        _paged(c, max_seqlen_q=most, max_seqlen_kv=most, scale=scale, window=(left, 0))
        p = seen.pop()
        assert (p.seqlen_q, p.seqlen_kv, p.softmax_scale, p.window_left) == (n, n, n / 4, n + 8)
    eps = torch.tensor(0.25)
    for e in (0.25, 0.5):
        eps.fill_(e)
        sdpa.sdpa_qk_norm_rope(c["q"], c["k"], c["w"], c["w"], eps=eps)
        assert seen.pop().eps == e


@pytest.mark.parametrize("kw,shift", [
    (dict(), 0),                                                      # one cache for both
    (dict(), 8), (dict(), -8), (dict(), 64), (dict(), 16 * 256 - 64),  # V begins inside K's rows, or ends in them
    (dict(), 16 * 256),                                               # V's pages are K's next ones
    (dict(k_page_stride=2 * 16 * 256, v_page_stride=2 * 16 * 256), 16 * 256 - 8),
    (dict(k_page_stride=2 * 16 * 256, v_page_stride=2 * 16 * 256), 16 * 256 + 8),
    (dict(k_page_stride=2 * 16 * 256, v_page_stride=3 * 16 * 256), 16 * 256),
    (dict(k_slot_stride=512, v_slot_stride=512, k_page_stride=8192, v_page_stride=8192), 128),
    (dict(num_heads_kv=1, num_pages=1, k_slot_stride=256, v_slot_stride=256), 120),
    (dict(num_heads_kv=1, num_pages=1, k_slot_stride=256, v_slot_stride=256), -120),
])
def test_append_refuses_caches_that_share_values(kw, shift):
    base = dict(num_heads_q=8, num_pages=50)
    p = paged_problem(**{**base, **kw})
    addr = [BASE, BASE + M, BASE + 2 * M, None, None, None, None, None, BASE + 8 * M, BASE + 8 * M + 2 * shift, BASE + 30 * M,
            BASE + 31 * M, BASE + 32 * M]
    assert sdpa.sdpa_check_paged(p) == 0
    assert sdpa.lib().sdpa_paged_append(ctypes.byref(p), None, *[PTR(x) for x in addr], None) == 4


@pytest.mark.parametrize("kw", [dict(k_page_stride=8 * 256), dict(v_page_stride=256),
                                dict(k_slot_stride=128, k_head_stride=1024, v_slot_stride=128, v_head_stride=1024)])
def test_append_refuses_a_cache_whose_rows_share_values(kw):
    p = paged_problem(**kw)
    addr = [BASE, BASE + M, BASE + 2 * M, None, None, None, None, None, BASE + 8 * M, BASE + 20 * M, BASE + 30 * M,
            BASE + 31 * M, BASE + 32 * M]
    assert sdpa.sdpa_check_paged(p) == 0
    assert sdpa.lib().sdpa_paged_append(ctypes.byref(p), None, *[PTR(x) for x in addr], None) == 4


@pytest.mark.parametrize("kw", [dict(window=(2 ** 32, -1)), dict(window=(2 ** 31, 0)), dict(window=(-2 ** 40, -1)),
                                dict(max_seqlen_q=2 ** 32 + 2), dict(max_seqlen_kv=2 ** 32 + 16), dict(max_seqlen_kv=2 ** 31)])
def test_sizes_beyond_32_bits_are_refused(monkeypatch, kw):
    """The struct's fields would keep their low bits only: a window of 2^32 became one of 0."""
    monkeypatch.setattr(sdpa, "_refuse_cpu", lambda t: None)
    monkeypatch.setattr(sdpa, "_launch", lambda name, device, *args: None)
    with pytest.raises(ValueError, match="32 bits"):
        _paged(_batch(), **kw)


def test_a_table_of_more_keys_than_a_sequence_can_have(monkeypatch):
    """The default bound of the lengths is what the table holds, but never more than the library serves (2^30)."""
    seen = []
    monkeypatch.setattr(sdpa, "_refuse_cpu", lambda t: None)
    monkeypatch.setattr(sdpa, "_launch", lambda name, device, *args: seen.append(args[0]._obj))
    c = _batch()
    _paged(c)
    assert seen.pop().seqlen_kv == 4 * 16
    meta = lambda t: (t.shape, t.stride(), t.dtype, t.device)  # noqa: E731
    q, lens, cu = meta(c["q"]), meta(c["lens"]), meta(c["cu"])
    for page, cols in ((1 << 20, 1025), (1 << 20, 4096), (1 << 19, 1 << 13)):
        cache = (torch.Size((1, page, 2, 128)), (page * 256, 256, 128, 1), torch.bfloat16, c["q"].device)
        table = (torch.Size((3, cols)), (cols, 1), torch.int32, c["q"].device)
        p, need = sdpa._paged_plan(q, cache, cache, table, lens, cu, 2, None, "nhd", "causal_br", -1, -1, None, None, None)
        assert p.seqlen_kv == 1 << 30 and sdpa.sdpa_check_paged(p) == 0 and need > 0


def test_a_right_bound_without_a_causal_mask_is_refused(monkeypatch):
    """sdpa_fwd hides the keys right of the diagonal then; the paged call has no such mask and saw them all."""
    seen = []
    monkeypatch.setattr(sdpa, "_refuse_cpu", lambda t: None)
    monkeypatch.setattr(sdpa, "_launch", lambda name, device, *args: seen.append(name))
    for window in ((-1, -1), (-1, 0), (3, 0)):
        _paged(_batch(), window=window)
    _paged(_batch(), mask="none")
    assert len(seen) == 4
    with pytest.raises(ValueError, match="causal_br"):
        _paged(_batch(), mask="none", window=(-1, 0))
