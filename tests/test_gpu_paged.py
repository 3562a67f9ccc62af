"""Attention over a paged cache against the 64-bit reference.

Tolerances, before the first run. S: products of 16-bit values are exact, their
fp32 sum over D in groups of 16 is off by at most (D / 8) 2^-23 of sum |q||k|
scale =: a. Exponents and exponentials add 2^-19 relative at the magnitudes
here. P is rounded to 16 bits (u, half a step; fp16 below 2^-14: 2^-25, with a
row sum of at least 1 and n keys), O once more:
  |O - O'| <= (u + 2 (D/8) 2^-23 a + 2^-19) sum p|v| + u |O| + [fp16] (n + 1) 2^-25 max|v|
  |LSE - LSE'| <= 2 (D/8) 2^-23 a + 2^-19 (1 + |LSE|)
Rows without keys are exactly 0 and -inf.
"""
import numpy as np
import pytest
import torch

import paged_ref as ref
import scaled_dot_product_02_gb300 as sdpa

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def case(new, total, hq=8, hkv=2, d=128, dv=None, page=16, order="nhd", dtype=BF, pad=0, seed=0, poison=True, std=1.0,
         max_kv=0):
    """A batch on the CPU and the GPU; slots that hold no key of their sequence are NaN. max_kv: the bound given for
    the lengths, when larger than they are."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dv = dv or (128 if d == 192 else d)
    n = lambda *s: (torch.randn(*s, generator=g) * std).to(dtype)  # noqa: E731
    table, pages = ref.make_pages(rng, total, page, cols=max(1, -(-max(max_kv, max(total)) // page)))
    kc, vc = n(pages, page, hkv, d), n(pages, page, hkv, dv)
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, k in enumerate(total):
        p = np.arange(k)
        used[torch.from_numpy(table[b, p // page].astype(np.int64)), torch.from_numpy(p % page)] = True
    if poison:
        kc[~used] = float("nan")
        vc[~used] = float("nan")
    if order == "hnd":
        kc, vc = kc.transpose(1, 2).contiguous(), vc.transpose(1, 2).contiguous()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = n(int(sum(new)) + pad, hq, d)
    c = dict(q=q, kc=kc, vc=vc, table=table, cu=cu, lens=np.array(total, dtype=np.int32), page=page, order=order,
             max_q=max(max(new), 1), max_kv=max(max(total), max_kv, 1), scale=d ** -0.5, dtype=dtype)
    c["dev"] = [q.cuda(), kc.cuda(), vc.cuda()] + [torch.from_numpy(x).cuda() for x in (table, c["lens"], cu)]
    return c


def call(c, causal=True, window=-1, **kw):
    return sdpa.sdpa_paged_fwd(*c["dev"], max_seqlen_q=c["max_q"], max_seqlen_kv=c["max_kv"], cache_layout=c["order"],
                               mask="causal_br" if causal else "none", window=(window, -1), scale=c["scale"], **kw)


def check(c, o, lse, causal=True, window=-1):
    d = c["q"].shape[-1]
    live = int(c["cu"][-1])
    want, want_l, pv, mag = ref.paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], c["page"],
                                                c["order"], causal, window, c["scale"])
    o, lse, want, want_l, pv, mag = (x[:live] for x in (o.cpu().double(), lse.cpu().double(), want, want_l, pv, mag))
    empty = want_l == -np.inf
    assert bool((lse[empty] == -np.inf).all()) and not bool(o[empty].any())
    assert bool(torch.isfinite(lse[~empty]).all())
    u = ref.U[c["dtype"]]
    s_err = 2 * (d / 8) * 2.0 ** -23 * mag
    tol = (u + s_err + 2.0 ** -19)[..., None] * pv + u * want.abs() + 1e-12
    if c["dtype"] == HF:
        vmax = c["vc"].float().nan_to_num().abs().max().item()
        tol = tol + (c["max_kv"] + 1) * 2.0 ** -25 * vmax
    err = (o - want).abs()
    assert bool((err <= tol)[~empty].all()), f"O: worst {(err / tol)[~empty].max().item():.2f} of the tolerance"
    err, tol = (lse - want_l)[~empty].abs(), (s_err + 2.0 ** -19 * (1 + want_l.abs()))[~empty]
    assert bool((err <= tol).all()), f"LSE: worst {(err / tol).max().item():.2f} of the tolerance"
    assert sdpa.sdpa_get_device_error() == 0


BATCHES = {
    "one": ([1], [1]),
    "one_long": ([1], [1500]),
    "tile": ([1, 1, 1, 1], [127, 128, 129, 256]),
    "ragged": ([1] * 9, [1, 2, 15, 16, 17, 300, 1000, 64, 513]),
    "spec": ([5, 0, 1, 3, 2], [5, 7, 130, 400, 2]),
    "chunk": ([70, 1, 33], [70, 90, 700]),
    "short_cache": ([4, 3, 2], [2, 0, 2]),       # more new tokens than keys: rows in front of the cache see none
}
DIMS = [(128, 16, "nhd"), (192, 48, "hnd"), (256, 64, "hnd"), (512, 128, "nhd"), (128, 256, "hnd"), (256, 32, "nhd")]


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("d,page,order", DIMS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_lengths(batch, d, page, order, dtype):
    c = case(*BATCHES[batch], d=d, page=page, order=order, dtype=dtype, pad=2)
    out = torch.full((c["q"].shape[0], 8, c["vc"].shape[-1]), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((c["q"].shape[0], 8), 9.0, device="cuda")
    o, l = call(c, out=out, lse=lse)
    assert o is out and l is lse
    check(c, o, l)
    assert bool((out[-2:] == 9).all()) and bool((lse[-2:] == 9).all())  # rows behind the last sequence


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (14, 2), (32, 8), (16, 1), (40, 1), (80, 1), (33, 1), (96, 2), (200, 1)])
@pytest.mark.parametrize("d", [128, 192, 256, 512])
def test_head_groups(hq, hkv, d):
    for new, total in (([1, 1, 1], [5, 200, 700]), ([9, 2], [140, 300])):
        c = case(new, total, hq=hq, hkv=hkv, d=d, page=32)
        check(c, *call(c))


@pytest.mark.parametrize("window", [0, 5, 127, 128, 300, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("d,page,order", DIMS[:4])
def test_windows(window, d, page, order):
    for name in ("ragged", "chunk", "spec"):
        c = case(*BATCHES[name], d=d, page=page, order=order)
        check(c, *call(c, window=window), window=window)


@pytest.mark.parametrize("d", [128, 256])
def test_pages_behind_a_window_are_never_read(d):
    window, page = 40, 16
    c = case([1, 3, 1], [1000, 333, 30], d=d, page=page)
    table = c["dev"][3].clone()
    kc, vc = c["dev"][1].clone(), c["dev"][2].clone()
    for b, (q, n) in enumerate(((1, 1000), (3, 333))):
        first = n - q - window
        table[b, :first // page] = 2 ** 31 - 1           # freed: not a page
        for s in range(first % page):                     # slots of the first kept page in front of the window
            p = int(c["table"][b, first // page])
            kc[p, s], vc[p, s] = float("nan"), float("inf")
    c["dev"][3], c["dev"][1], c["dev"][2] = table, kc, vc
    check(c, *call(c, window=window), window=window)


@pytest.mark.parametrize("d", [128, 192, 512])
@pytest.mark.parametrize("name", ["ragged", "spec", "chunk"])
def test_no_mask(d, name):
    c = case(*BATCHES[name], d=d, dtype=HF)
    check(c, *call(c, causal=False), causal=False)


def test_scores_of_any_size():
    for std in (0.02, 4.0):  # flat rows; rows where one key takes all and the running maximum moves often
        c = case([1, 2, 40], [900, 1400, 500], std=std)
        c["scale"] = 0.3
        check(c, *call(c))
    c = case([1, 2], [300, 500])
    c["scale"] = 0.0
    check(c, *call(c))


def test_rising_scores_move_the_maximum_every_tile():
    c = case([2], [1200], hq=4, hkv=1)
    q, kc = c["q"], c["kc"]
    q.fill_(1.0)
    for pos in range(1200):
        kc[int(c["table"][0, pos // 16]), pos % 16] = float(pos // 100)  # scores climb by 11 every 100 keys
    c["dev"][0], c["dev"][1] = q.cuda(), kc.cuda()
    check(c, *call(c))


@pytest.mark.parametrize("name", ["one_long", "ragged", "chunk"])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_reproducible_and_independent_of_the_split(name, d):
    c = case(*BATCHES[name], d=d)
    a, b = call(c), call(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    try:
        for cap in (1, 2, 3, 7, 50):  # workers of either kernel
            sdpa.sdpa_debug_set_max_ctas(cap)
            check(c, *call(c))
    finally:
        sdpa.sdpa_debug_set_max_ctas(0)


def test_strided_q_and_pages_that_hold_k_and_v():
    c = case([1, 4], [100, 260], poison=False)
    q, kc, vc = c["dev"][:3]
    both = torch.stack([kc, vc], dim=1)
    wide = torch.randn(q.shape[0], 8 * 128 + 512, device="cuda").to(BF)
    wide[:, :1024] = q.flatten(1)
    c["dev"][0] = wide[:, :1024].unflatten(1, (8, 128))
    c["dev"][1], c["dev"][2] = both[:, 0], both[:, 1]
    tab = torch.full((2, 40), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    tab[:, :c["table"].shape[1]] = c["dev"][3]
    c["dev"][3] = tab[:, :c["table"].shape[1]]
    check(c, *call(c))


def test_offsets_beyond_32_bits():
    """Pages whose elements start beyond 2^31 (and bytes beyond 2^32)."""
    pages, page, hkv, d = 140000, 64, 2, 128
    kc = torch.empty(pages, page, hkv, d, dtype=BF, device="cuda")
    vc = torch.empty(pages, page, hkv, d, dtype=BF, device="cuda")
    assert kc.numel() > 2 ** 31
    c = case([1, 2], [100, 200], page=page, hkv=hkv)
    ids = np.array([[139999, 131072, -1, -1], [139000, 5, 135000, 131071]], dtype=np.int32)
    k_new, v_new = torch.randn(3, hkv, d, device="cuda").to(BF), torch.randn(3, hkv, d, device="cuda").to(BF)
    for b in range(2):
        for j in range(c["table"].shape[1]):
            if ids[b, j] >= 0 and c["table"][b, j] >= 0:
                kc[int(ids[b, j])], vc[int(ids[b, j])] = c["dev"][1][int(c["table"][b, j])], c["dev"][2][int(c["table"][b, j])]
    tab = torch.from_numpy(ids).cuda()
    sdpa.sdpa_paged_append(k_new, v_new, kc, vc, tab, c["dev"][4], c["dev"][5])
    for row, pg, slot, _, _ in ref.token_places(c["cu"], c["lens"], page, c["table"]).T:
        c["kc"][pg, slot], c["vc"][pg, slot] = k_new[row].cpu(), v_new[row].cpu()
    c["dev"][1], c["dev"][2], c["dev"][3] = kc, vc, tab
    check(c, *call(c))


def test_bad_metadata_is_refused_on_the_device():
    c = case([1, 3], [200, 77], poison=False)
    q, kc, vc, tab, lens, cu = c["dev"]
    out, lse = torch.full((4, 8, 128), 3.0, dtype=BF, device="cuda"), torch.full((4, 8), 3.0, device="cuda")
    f = lambda t=tab, n=lens, u=cu, **kw: sdpa.sdpa_paged_fwd(  # noqa: E731
        q, kc, vc, t, n, u, max_seqlen_q=kw.get("mq", 3), max_seqlen_kv=kw.get("mk", 200), out=out, lse=lse)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in (dict(n=i32(201, 77)), dict(n=i32(200, -1)), dict(u=i32(0, 1, 5)), dict(u=i32(0, 2, 1)), dict(u=i32(1, 2, 4)),
                dict(u=i32(0, -1, 3)), dict(mq=2), dict(mk=199)):
        f(**bad)
        assert sdpa.sdpa_get_device_error() == 6, bad
        assert bool((out == 3).all()) and bool((lse == 3).all())
    for page in (-1, kc.shape[0], 2 ** 31 - 1):
        t = tab.clone()
        t[0, 3] = page
        f(t=t)
        assert sdpa.sdpa_get_device_error() == 10
    f()
    check(c, out, lse)


def test_captured_calls_follow_the_lengths_and_share_a_workspace():
    c = case([1] * 4, [700, 30, 260, 129])
    e = case([3, 1], [500, 90], d=256, page=32, seed=3)
    ws = torch.empty(sdpa.PAGED_WORKSPACE_MAX, dtype=torch.uint8, device="cuda")
    call(c, workspace=ws), call(e, workspace=ws)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        a = call(c, workspace=ws)
    with torch.cuda.graph(g2):
        b = call(e, workspace=ws)
    for lens in ([700, 30, 260, 129], [1, 2, 3, 4], [513, 16, 128, 100]):
        c["lens"] = np.array(lens, dtype=np.int32)
        c["dev"][4].copy_(torch.from_numpy(c["lens"]))
        ws.fill_(255)
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        check(c, *a)
        check(e, *b)


def test_two_calls_at_once_on_two_streams():
    c = case([60, 1, 5], [900, 2000, 300], pad=1)
    e = case([1, 3, 200], [1500, 700, 800], d=256, page=64, order="hnd")
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [(call(c, stream=streams[0]), call(e, stream=streams[1])) for _ in range(10)]
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[0][:-1], got[0][0][0][:-1]) and torch.equal(b[0], got[0][1][0])
    check(c, *got[-1][0])
    check(e, *got[-1][1])


def test_a_mixed_call_is_timed_and_follows_other_work():
    """Events around its launches, which then run strictly in turn; and calls back to back on one workspace."""
    c = case([90, 1, 0, 2], [500, 1200, 7, 300])
    ws = torch.empty(sdpa.PAGED_WORKSPACE_MAX, dtype=torch.uint8, device="cuda")
    sdpa.sdpa_profile_begin()
    a = call(c, workspace=ws)
    kinds = sdpa.sdpa_profile_end()
    assert kinds["paged"][1] >= 1 and kinds["paged"][0] > 0
    check(c, *a)
    keep = [call(c, workspace=ws) for _ in range(20)]
    assert all(torch.equal(x[0], a[0]) and torch.equal(x[1], a[1]) for x in keep)


def test_another_stream():
    c = case([1, 2], [300, 400])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = call(c, stream=side)
    side.synchronize()
    check(c, o, lse)


def test_an_empty_batch_and_empty_sequences():
    c = case([0, 0], [5, 9])
    o, lse = call(c)
    assert o.shape == (0, 8, 128) and lse.shape == (0, 8)
    c = case([0, 0], [5, 9], pad=3)
    out, lse = torch.full((3, 8, 128), 2.0, dtype=BF, device="cuda"), torch.full((3, 8), 2.0, device="cuda")
    call(c, out=out, lse=lse)
    assert bool((out == 2).all()) and bool((lse == 2).all()) and sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("d,page", [(128, 16), (256, 64), (512, 128)])
@pytest.mark.parametrize("window", [-1, 777])
def test_many_tiles_and_many_items_per_cta(d, page, window):
    """Every ring slot is taken again and again before the tile whose unseen values are cleared."""
    c = case([150, 1, 60, 7], [3001, 2777, 1900, 2050], hq=16, hkv=4, d=d, page=page)
    check(c, *call(c, window=window), window=window)


@pytest.mark.parametrize("d,page,order", [(128, 64, "nhd"), (192, 16, "nhd"), (256, 256, "hnd"), (512, 32, "nhd")])
@pytest.mark.parametrize("window", [-1, 100])
def test_long_chunks_and_single_tokens_in_one_batch(d, page, order, window):
    """Sequences on both sides of the cut between the two kernels, one and many items per CTA."""
    c = case([300, 1, 0, 17, 700, 16, 1], [300, 900, 30, 800, 1500, 16, 1], hq=16, hkv=4, d=d, page=page, order=order, pad=3)
    check(c, *call(c, window=window), window=window)
    c = case([1111], [2000], hq=8, hkv=2, d=d, page=page, order=order, dtype=HF)
    check(c, *call(c, window=window), window=window)


@pytest.mark.parametrize("d", [128, 256])
def test_items_enough_for_the_ticket_order(d):
    c = case([600, 1, 333], [700, 50, 1300], hq=64, hkv=32, d=d, page=64)
    check(c, *call(c))
    check(c, *call(c, window=200), window=200)


@pytest.mark.parametrize("d", [128, 192])
@pytest.mark.parametrize("n", [3, 128, 129, 200])
def test_ticket_order_of_many_sequences(d, n):
    """Sorted by their keys up to 128 sequences, in their own order above; equal lengths and empty ones among them."""
    rng = np.random.default_rng(n)
    new = rng.integers(0, 60, n)
    new[:2] = 59
    total = np.maximum(new, rng.integers(0, 4, n) * 70 + 5)
    c = case(new.tolist(), total.tolist(), hq=8, hkv=4, d=d, page=16, pad=2)
    check(c, *call(c))


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (128, 3, 3), (192, 8, 2), (256, 16, 4), (512, 4, 1)])
@pytest.mark.parametrize("new,total", [([300], [2000]), ([700, 40, 33, 500], [700, 41, 3000, 900]), ([40] * 60, [50] * 60),
                                       ([64, 200, 0, 3], [10, 0, 0, 1000])])
def test_the_last_items_cut_into_shares(d, hq, hkv, new, total):
    """Long contexts (by their bound) of few items: with no, one and several rounds of whole items before the rest."""
    c = case(new, total, hq=hq, hkv=hkv, d=d, page=64, max_kv=33000 if d == 128 else 7000)
    a, b = call(c), call(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the shares do not depend on who takes them
    check(c, *a)
    try:
        for cap in (1, 2, 5, 33):
            sdpa.sdpa_debug_set_max_ctas(cap)
            check(c, *call(c))
    finally:
        sdpa.sdpa_debug_set_max_ctas(0)
    check(c, *call(c, window=150), window=150)
    check(c, *call(c, causal=False), causal=False)


def test_a_large_batch():
    rng = np.random.default_rng(5)
    total = rng.integers(1, 200, 700)
    c = case([1] * 700, total.tolist(), hq=4, hkv=2)
    check(c, *call(c))


def test_agrees_with_the_contiguous_forward():
    """One sequence whose pages are in order is the contiguous bottom-right problem."""
    n, m = 384, 100
    c = case([m], [n], page=128, poison=False)
    c["table"][:] = np.arange(3)
    c["dev"][3].copy_(torch.from_numpy(c["table"]))
    o, lse = call(c)
    q, kc, vc = c["dev"][:3]
    o2, lse2 = sdpa.sdpa_fwd(q[None], kc[:3].reshape(1, n, 2, 128), vc[:3].reshape(1, n, 2, 128), mask="causal_br")
    check(c, o, lse)
    check(c, o2[0], lse2)


def test_a_step_of_a_model():
    """Norm + rotation + append + attention in turn, prompt then single tokens, equals attention over all keys at once."""
    hq, hkv, d, page, n = 8, 2, 128, 16, 90
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(n, (hq + 2 * hkv) * d, device="cuda", generator=g).to(BF)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    wq, wk = (1 + 0.1 * torch.randn(2, d, device="cuda", generator=g)).to(BF)
    table = ref.angles_table(n, d).cuda()
    kc = torch.full((8, page, hkv, d), float("nan"), dtype=BF, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    ids = torch.tensor([[6, 2, 7, 0, 3, 5]], dtype=torch.int32, device="cuda")
    outs, lses, at = [], [], 0
    for m in (70, 1, 1, 17, 1):
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        lens = torch.tensor([at + m], dtype=torch.int32, device="cuda")
        qo = sdpa.sdpa_paged_append(k[at:at + m], v[at:at + m], kc, vc, ids, lens, cu, q=q[at:at + m], q_weight=wq,
                                    k_weight=wk, cos_sin=table)
        o, lse = sdpa.sdpa_paged_fwd(qo, kc, vc, ids, lens, cu, max_seqlen_q=m)
        outs.append(o)
        lses.append(lse)
        at += m
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    qr, kr = sdpa.sdpa_qk_norm_rope(q, k, wq, wk, table, pos)
    c = dict(q=qr.cpu(), kc=kr.cpu()[None], vc=v.cpu()[None], table=np.zeros((1, 1), np.int32), cu=np.array([0, n]),
             lens=np.array([n]), page=n, order="nhd", max_kv=n, scale=d ** -0.5, dtype=BF)
    check(c, torch.cat(outs), torch.cat(lses))


@pytest.mark.parametrize("d,order", [(128, "nhd"), (192, "hnd"), (256, "nhd"), (512, "hnd")])
def test_every_access_is_inside_the_buffers(d, order):
    c = case([1, 0, 5, 40], [700, 3, 90, 300], d=d, order=order, pad=1, dtype=HF)
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        o, lse = call(c)
        assert sdpa.sdpa_debug_address_report()[0] == 0
        assert sdpa.sdpa_get_device_error() == 0
    check(c, o, lse)


@pytest.mark.parametrize("capture", [False, True])
def test_memory_of_a_call_on_another_stream(monkeypatch, capture):
    """The workspace of a call is not handed out again on the calling stream, and its outputs outlive a use there."""
    c = case([3, 1, 5], [900, 400, 2000])
    want = call(c)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(here)
    seen, launch = [], sdpa._launch
    monkeypatch.setattr(sdpa, "_launch", lambda name, device, *a: (seen.append((a[-2], a[-1])), launch(name, device, *a)))
    o, lse = call(c, stream=side)
    (at, size), = seen
    again = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() + size <= at or at + size <= x.data_ptr() for x in again)
    assert torch.cuda.current_stream() == here
    here.wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    if capture:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            inner = torch.cuda.Stream()
            inner.wait_stream(torch.cuda.current_stream())
            o, lse = call(c, stream=inner)
            torch.cuda.current_stream().wait_stream(inner)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [128, 192, 256, 512])
@pytest.mark.parametrize("new,window", [([2], -1), ([5, 1], -1), ([40], -1), ([33, 20], 7000), ([1, 16, 3], -1)])
def test_few_items_of_many_parts(d, new, window):
    """Items that most of the CTAs share: their parts are joined by all the cuts inside them."""
    total = [9001, 7777, 8200][:len(new)]
    c = case(new, total, hq=9, hkv=1 if d != 192 else 3, d=d, page=32, seed=31, max_kv=33000 if d == 128 else 0)
    o, lse = call(c, window=window)
    check(c, o, lse, window=window)
    again = call(c, window=window)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def bare_call(c, monkeypatch, **kw):
    """The problem struct of a call, which is not made."""
    seen = []
    with monkeypatch.context() as m:
        m.setattr(sdpa, "_launch", lambda name, device, *a: seen.append(a[0]._obj))
        call(c, **kw)
    return seen[0]


# (new, total, bound of the lengths, window): shares cut or not, in the rows kernel, the chunk kernel and both
EXACT = {
    "whole_items": ([1] * 80, [40 + 3 * i for i in range(80)], 512, -1),
    "split_items": ([1] * 80, [40 + 3 * i for i in range(80)], 513, -1),
    "small_window": ([1] * 80, [1000 + 3 * i for i in range(80)], 4000, 100),
    "whole_chunks": ([40] * 30, [300 + i for i in range(30)], 512, -1),
    "cut_chunks": ([40, 33], [700, 300], 33000, -1),
    "mixed_whole": ([1, 40, 0, 17, 2], [400, 90, 7, 300, 512], 512, -1),
    "mixed_cut": ([1, 40, 0, 17, 2], [4000, 90, 7, 300, 512], 33000, -1),
}


@pytest.mark.parametrize("name", EXACT)
@pytest.mark.parametrize("d", [128, 192, 256, 512])
def test_a_workspace_of_the_reported_size_is_enough(name, d, monkeypatch):
    """Nothing in front of the workspace or behind it is written."""
    new, total, max_kv, window = EXACT[name]
    c = case(new, total, hq=16, hkv=8, d=d, max_kv=max_kv)
    need = sdpa.sdpa_paged_fwd_workspace_size(bare_call(c, monkeypatch, window=window))
    edge = 1 << 16
    whole = torch.full((edge + need + edge,), 0xA5, dtype=torch.uint8, device="cuda")
    check(c, *call(c, window=window, workspace=whole[edge:edge + need]), window=window)
    assert bool((whole[:edge] == 0xA5).all()) and bool((whole[edge + need:] == 0xA5).all())


@pytest.mark.parametrize("name", EXACT)
@pytest.mark.parametrize("d", [128, 192, 256, 512])
def test_every_access_is_inside_a_workspace_of_the_reported_size(name, d):
    new, total, max_kv, window = EXACT[name]
    c = case(new, total, hq=16, hkv=8, d=d, max_kv=max_kv)
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        o, lse = call(c, window=window)
        assert sdpa.sdpa_debug_address_report()[0] == 0
        assert sdpa.sdpa_get_device_error() == 0
    check(c, o, lse, window=window)


@pytest.mark.parametrize("d,page,order", DIMS[:4])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal,window", [(True, -1), (True, 33), (False, -1)])
def test_a_scale_of_zero(d, page, order, dtype, causal, window):
    """All visible keys weigh the same, hidden ones nothing: single tokens, chunks, both in one batch, and the last items
    cut into shares."""
    for new, total, max_kv in (([1, 2], [300, 501], 0), ([70, 1, 33], [70, 90, 701], 0), ([300, 41], [911, 333], 33000)):
        c = case(new, total, d=d, page=page, order=order, dtype=dtype, max_kv=max_kv)
        c["scale"] = 0.0
        check(c, *call(c, causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("d", [128, 192])
@pytest.mark.parametrize("n", [3, 31, 32, 33, 64, 65])
@pytest.mark.parametrize("hkv", [2, 4])
@pytest.mark.parametrize("cut", [False, True])
def test_ticket_order_on_both_sides_of_sorting(d, n, hkv, cut):
    """Sorted by their keys up to 32 sequences, in their own order above, 32 of them a step; equal lengths and empty
    sequences among them, whole items alone or the last ones cut into shares."""
    rng = np.random.default_rng(n)
    new = rng.integers(0, 60, n)
    new[:2] = 59
    total = np.maximum(new, rng.integers(0, 4, n) * 170 + 5)
    c = case(new.tolist(), total.tolist(), hq=8, hkv=hkv, d=d, page=16, pad=2, max_kv=33000 if cut else 0)
    a, b = call(c), call(c)
    live = int(c["cu"][-1])
    assert torch.equal(a[0][:live], b[0][:live]) and torch.equal(a[1][:live], b[1][:live])
    check(c, *a)


@pytest.mark.parametrize("d,items,tiles,cut", [
    (d, *x) for d in (192, 256, 512) for x in (
        (24, 15, False), (24, 16, True), (72, 27, False), (72, 28, True), (88, 47, False), (88, 48, True), (104, 95, False),
        (104, 96, True), (136, 300, False), (176, 47, False), (176, 48, True), (248, 95, False), (248, 96, True),
        (288, 300, False), (512, 48, True), (576, 300, False), (912, 300, False))
] + [(128, *x) for x in ((24, 16, False), (24, 17, True), (72, 35, False), (72, 36, True), (88, 255, False), (88, 256, True),
                         (136, 300, False), (168, 256, True), (256, 256, True), (288, 300, False), (512, 300, False))])
def test_which_chunks_are_cut(d, items, tiles, cut, monkeypatch):
    """Both sides of every border of the rule, by the number of items and the bound of the lengths; whole items need no
    more than the counters' 256 bytes of workspace."""
    heads = 4 if d == 512 else 8  # at 512 an item has half of the value columns
    n = items // 8
    rng = np.random.default_rng(items + tiles)
    total = rng.integers(70, 400, n)
    total[0] = 1900
    c = case([70] * n, total.tolist(), hq=heads, hkv=heads, d=d, page=32, max_kv=tiles * 128)
    assert (sdpa.sdpa_paged_fwd_workspace_size(bare_call(c, monkeypatch)) > 256) == cut
    a, b = call(c), call(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(c, *a)
