"""The 8-bit paged cache: rows quantised as they are written, read back, and
attention over them, against their definitions in 64 bits.

Tolerances, before the first run.
Append without a norm: codes and scale bytes are functions of the 16-bit row
alone, and equal. With it, K comes from fp32 values off by 2^-19 of the
magnitudes that enter them (test_gpu_norm_rope.py): the stored value is within
half a step of E4M3 (2^-4 of the value, and half of 2^-9 2^e below 2^-6 2^e) plus
that, doubled where the exponent differs from the exact one by one, which it may
only where the row's largest magnitude lies within 2^-18 of a border.
Read back: exact.
Attention. Products of a code and a part of q are exact; the fp32 sums over D
are off by at most (D / 8) 2^-23 of a := sum |q||k| scale for each of q's parts,
which sum to less than 1.25 a. Exponents and exponentials 2^-19. P is held to
2^-10 of itself, with a step of 2^-28 of the row's largest weight 2^ev p below
which n keys may vanish, each of a value of at most 448 2^ev:
  |O - O'| <= (2^-10 + 2.5 (D/8) 2^-23 a + 2^-19) sum p|v| + u |O| + (n + 1) 2^-27 max|v|
  |LSE - LSE'| <= 2.5 (D/8) 2^-23 a + 2^-19 (1 + |LSE|)
Rows without keys are exactly 0 and -inf.
"""
import numpy as np
import pytest
import torch

import fp8_ref
import paged_ref as ref
import scaled_dot_product_02_gb300 as sdpa
from test_gpu_paged import BATCHES, DIMS

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def ordered(x, order):
    """[pages, slots, heads(, width)] in the cache's order."""
    return x if order == "nhd" else x.transpose(1, 2).contiguous()


def cache(rng, g, pages, page, hkv, width, dtype, spread):
    """Quantised random rows (CPU, nhd): normal values times a token's magnitude 2^(-spread .. spread)."""
    x = torch.randn(pages, page, hkv, width, generator=g)
    x = x * torch.exp2(torch.from_numpy(rng.uniform(-spread, spread, (pages, page, hkv, 1))).float())
    return fp8_ref.quantise(x, dtype)


def case(new, total, hq=8, hkv=2, d=128, dv=None, page=16, order="nhd", dtype=BF, pad=0, seed=0, poison=True, spread=2.0,
         max_kv=0, q_std=1.0):
    """A batch; slots that hold no key of their sequence have NaN codes and any scale byte."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dv = dv or (128 if d == 192 else d)
    table, pages = ref.make_pages(rng, total, page, cols=max(1, -(-max(max_kv, max(total)) // page)))
    kc, ks = cache(rng, g, pages, page, hkv, d, dtype, min(spread, 3.0))
    vc, vs = cache(rng, g, pages, page, hkv, dv, dtype, spread)
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, k in enumerate(total):
        p = np.arange(k)
        used[torch.from_numpy(table[b, p // page].astype(np.int64)), torch.from_numpy(p % page)] = True
    if poison:
        for codes, scale in ((kc, ks), (vc, vs)):
            codes[~used] = torch.from_numpy(rng.choice([127, 255, 126], (int((~used).sum()), 1, 1)).astype(np.uint8))
            scale[~used] = torch.from_numpy(rng.integers(0, 256, (int((~used).sum()), 1)).astype(np.uint8))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = (torch.randn(int(sum(new)) + pad, hq, d, generator=g) * q_std).to(dtype)
    c = dict(q=q, kc=fp8_ref.decode(kc, ks), vc=fp8_ref.decode(vc, vs), table=table, cu=cu, lens=np.array(total, dtype=np.int32),
             page=page, order=order, max_q=max(max(new), 1), max_kv=max(max(total), max_kv, 1), scale=d ** -0.5, dtype=dtype)
    c["dev"] = [q.cuda()] + [ordered(x, order).cuda() for x in (kc, vc, ks, vs)]
    c["dev"] += [torch.from_numpy(x).cuda() for x in (table, c["lens"], cu)]
    return c


def call(c, causal=True, window=-1, **kw):
    kw = {"scale": c["scale"], "max_seqlen_q": c["max_q"], "max_seqlen_kv": c["max_kv"], **kw}
    return sdpa.sdpa_paged_fwd_fp8(*c["dev"], cache_layout=c["order"], mask="causal_br" if causal else "none",
                                   window=(window, -1), **kw)


def check(c, o, lse, causal=True, window=-1, scale=None):
    d, live = c["q"].shape[-1], int(c["cu"][-1])
    want, want_l, pv, mag = ref.paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], c["page"], "nhd",
                                                causal, window, c["scale"] if scale is None else scale)
    o, lse, want, want_l, pv, mag = (x[:live] for x in (o.cpu().double(), lse.cpu().double(), want, want_l, pv, mag))
    empty = want_l == -np.inf
    assert bool((lse[empty] == -np.inf).all()) and not bool(o[empty].any())
    assert bool(torch.isfinite(lse[~empty]).all())
    s_err = 2.5 * (d / 8) * 2.0 ** -23 * mag
    vmax = c["vc"][torch.isfinite(c["vc"])].abs().max().item() if c.get("vmax") is None else c["vmax"]
    tol = (2.0 ** -10 + s_err + 2.0 ** -19)[..., None] * pv + ref.U[c["dtype"]] * want.abs() + ref.TINY[c["dtype"]]
    tol = tol + (c["max_kv"] + 1) * 2.0 ** -27 * vmax
    err = (o - want).abs()
    assert bool((err <= tol)[~empty].all()), f"O: worst {(err / tol)[~empty].max().item():.2f} of the tolerance"
    err, tol = (lse - want_l)[~empty].abs(), (s_err + 2.0 ** -19 * (1 + want_l.abs()))[~empty]
    assert bool((err <= tol).all()), f"LSE: worst {(err / tol).max().item():.2f} of the tolerance"
    assert sdpa.sdpa_get_device_error() == 0


def used_vmax(c):
    """The largest value of V that a sequence holds (unused slots may hold larger ones)."""
    top = 0.0
    for b, n in enumerate(c["lens"]):
        p = np.arange(n)
        rows = c["vc"][torch.from_numpy(c["table"][b, p // c["page"]].astype(np.int64)), torch.from_numpy(p % c["page"])]
        top = max(top, rows.abs().max().item() if n else 0.0)
    return top


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("d,page,order", DIMS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_lengths(batch, d, page, order, dtype):
    c = case(*BATCHES[batch], d=d, page=page, order=order, dtype=dtype, pad=2)
    c["vmax"] = used_vmax(c)
    out = torch.full((c["q"].shape[0], 8, c["vc"].shape[-1]), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((c["q"].shape[0], 8), 9.0, device="cuda")
    o, l = call(c, out=out, lse=lse)
    assert o is out and l is lse
    check(c, o, l)
    assert bool((out[-2:] == 9).all()) and bool((lse[-2:] == 9).all())  # rows behind the last sequence


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (14, 2), (32, 8), (16, 1), (40, 1), (33, 1), (96, 2)])
@pytest.mark.parametrize("d", [128, 192, 256, 512])
def test_attention_head_groups(hq, hkv, d):
    for new, total in (([1, 1, 1], [5, 200, 700]), ([9, 2], [140, 300])):
        c = case(new, total, hq=hq, hkv=hkv, d=d, page=32)
        c["vmax"] = used_vmax(c)
        check(c, *call(c))


@pytest.mark.parametrize("window", [0, 5, 127, 128, 300, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("d,page,order", DIMS[:4])
def test_attention_windows(window, d, page, order):
    for name in ("ragged", "chunk", "spec"):
        c = case(*BATCHES[name], d=d, page=page, order=order)
        c["vmax"] = used_vmax(c)
        check(c, *call(c, window=window), window=window)


@pytest.mark.parametrize("d", [128, 256])
def test_pages_behind_a_window_are_never_read(d):
    window, page = 40, 16
    c = case([1, 3, 1], [1000, 333, 30], d=d, page=page)
    c["vmax"] = used_vmax(c)
    q, kc, vc, ks, vs, table = (x.clone() for x in c["dev"][:6])
    for b, (n, k) in enumerate(((1, 1000), (3, 333))):
        first = k - n - window
        table[b, :first // page] = 2 ** 31 - 1           # freed: not a page
        p = int(c["table"][b, first // page])
        for s in range(first % page):                     # slots of the first kept page in front of the window
            kc[p, s], vc[p, s], ks[p, s], vs[p, s] = 127, 127, 255, 255
    c["dev"][:6] = [q, kc, vc, ks, vs, table]
    check(c, *call(c, window=window), window=window)


@pytest.mark.parametrize("d", [128, 192, 512])
@pytest.mark.parametrize("name", ["ragged", "spec", "chunk"])
def test_attention_without_a_mask(d, name):
    c = case(*BATCHES[name], d=d, dtype=HF)
    c["vmax"] = used_vmax(c)
    check(c, *call(c, causal=False), causal=False)


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 8), (256, 8, 2), (192, 32, 2)])
def test_values_of_very_different_sizes(d, hq, hkv):
    """Tokens' values between 2^-30 and 2^30 of one another, larger ones behind smaller ones and the reverse: the running
    maximum counts the values' exponents in."""
    for seed in range(3):
        c = case([1, 2, 1], [900, 513, 300], hq=hq, hkv=hkv, d=d, spread=30.0, seed=seed)
        c["vmax"] = used_vmax(c)
        check(c, *call(c))


def test_rising_scores_and_a_sink():
    """Scores that rise from tile to tile move the maximum every time; a first key that outweighs all others by 2^20
    leaves them their share."""
    d, n = 128, 1300
    c = case([1], [n], hq=4, hkv=1, d=d, poison=False)
    q = torch.ones(1, 4, d).bfloat16()
    for kind in ("rise", "sink", "fall"):
        top = {"rise": np.linspace(0, 40, n), "fall": np.linspace(40, 0, n), "sink": np.where(np.arange(n) == 0, 14.0, 0.0)}[kind]
        k = torch.zeros(n, d)
        k[:, 0] = torch.from_numpy(top * d ** 0.5).float()
        codes, scale = fp8_ref.quantise(k, BF)
        p = np.arange(n)
        at = (torch.from_numpy(c["table"][0, p // 16].astype(np.int64)), torch.from_numpy(p % 16))
        kc, ks = c["dev"][1].cpu(), c["dev"][3].cpu()
        kc[at[0], at[1], 0], ks[at[0], at[1], 0] = codes, scale
        c["kc"], c["q"] = fp8_ref.decode(kc, ks), q
        c["dev"][0], c["dev"][1], c["dev"][3] = q.cuda(), kc.cuda(), ks.cuda()
        check(c, *call(c))


def test_scale_of_zero_and_large_queries():
    c = case([1, 3], [300, 77], d=128, q_std=200.0)
    c["vmax"] = used_vmax(c)
    check(c, *call(c, scale=0.0), scale=0.0)
    check(c, *call(c, scale=1e-3), scale=1e-3)
    c = case([1, 3], [300, 77], d=256, dtype=HF, q_std=2.0 ** -12)
    c["vmax"] = used_vmax(c)
    check(c, *call(c, scale=8.0), scale=8.0)


def test_not_finite():
    """A query with an infinity or NaN gives NaN in its rows alone; a NaN key where it is seen."""
    c = case([2, 1], [200, 130], hq=4, hkv=2, d=128)
    good, good_l = call(c)
    c["dev"][0] = c["dev"][0].clone()
    c["dev"][0][0, 1, 5], c["dev"][0][1, 2, 7] = float("inf"), float("nan")
    o, lse = call(c)
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    assert bool(torch.isnan(o[bad]).all()) and torch.equal(o[~bad], good[~bad]) and torch.equal(lse[~bad], good_l[~bad])
    assert not bool(torch.isfinite(lse[bad]).any())
    c = case([2], [200], hq=2, hkv=2, d=128)
    good, _ = call(c)
    p = int(c["table"][0, 199 // 16])
    c["dev"][1][p, 199 % 16, 1, 3] = 127  # the last token's key of head 1
    o, _ = call(c)
    assert bool(torch.isnan(o[1, 1]).all()) and torch.equal(o[:, 0], good[:, 0]) and torch.equal(o[0, 1], good[0, 1])


def test_one_page_many_sequences_and_bits():
    """Sequences that share pages; a sequence's result does not depend on its batch when its cuts do not, and a call
    repeats bit for bit."""
    c = case([1] * 5, [400] * 5, d=128)
    c["dev"][5] = c["dev"][5][:1].expand(5, -1).contiguous()
    c["dev"][0] = c["dev"][0][:1].expand(5, -1, -1).contiguous()
    a, b = call(c), call(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c["q"], c["table"] = c["dev"][0].cpu(), c["dev"][5].cpu().numpy()
    c["vmax"] = used_vmax(c)
    check(c, *a)


def test_refused_batches_and_pages():
    c = case([1, 2], [100, 50], d=128)
    out, lse = torch.full((3, 8, 128), 4.0, dtype=BF, device="cuda"), torch.full((3, 8), 4.0, device="cuda")
    for at, bad in ((6, [101, 50]), (6, [-1, 50]), (7, [0, 2, 1]), (7, [1, 2, 3]), (7, [0, 1, 4])):
        dev = list(c["dev"])
        dev[at] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        sdpa.sdpa_paged_fwd_fp8(*dev, max_seqlen_q=2, max_seqlen_kv=100, out=out, lse=lse)
        assert sdpa.sdpa_get_device_error() == 6
        assert bool((out == 4).all()) and bool((lse == 4).all())
    dev = list(c["dev"])
    dev[5] = dev[5].clone()
    dev[5][0, 2] = 10 ** 6
    sdpa.sdpa_paged_fwd_fp8(*dev, max_seqlen_q=2, max_seqlen_kv=100, out=out, lse=lse)
    assert sdpa.sdpa_get_device_error() == 10
    check(c, *call(c))


def test_empty_calls():
    c = case([1, 2], [100, 50], d=128)
    o, lse = sdpa.sdpa_paged_fwd_fp8(c["dev"][0][:0], *c["dev"][1:5], c["dev"][5][:0], c["dev"][6][:0], c["dev"][7][:1],
                                     max_seqlen_q=1)
    assert o.shape == (0, 8, 128) and lse.shape == (0, 8)
    c = case([0, 0, 3], [0, 20, 3], d=256)
    check(c, *call(c))


@pytest.mark.parametrize("d", [128, 256, 512])
def test_any_schedule(d):
    c = case([1, 5, 2, 1], [700, 300, 1, 129], d=d)
    c["vmax"] = used_vmax(c)
    try:
        for cap in (1, 3, 7):
            sdpa.sdpa_debug_set_max_ctas(cap)
            check(c, *call(c))
    finally:
        sdpa.sdpa_debug_set_max_ctas(0)


# ---------------------------------------------------------------- append

def write_batch(seed, new, total, page, hkv, d, dv, order, dtype, pad=0, hq=None, std=1.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    table, pages = ref.make_pages(rng, total, page)
    rows = sum(new) + pad
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    whole = (torch.randn(rows, (hq or 0) * d + hkv * (d + dv), generator=g) * std).to(dtype).cuda()
    at = (hq or 0) * d
    s = dict(k=whole[:, at:at + hkv * d].unflatten(1, (hkv, d)), v=whole[:, at + hkv * d:].unflatten(1, (hkv, dv)), table=table,
             cu=cu, lens=np.array(total, dtype=np.int32), page=page, order=order, dtype=dtype)
    if hq:
        s["q"] = whole[:, :at].unflatten(1, (hq, d))
    byte = lambda *x: torch.from_numpy(rng.integers(0, 256, x).astype(np.uint8)).cuda()  # noqa: E731
    heads = (pages, page, hkv) if order == "nhd" else (pages, hkv, page)
    s["caches"] = [byte(*heads, d), byte(*heads, dv), byte(*heads), byte(*heads)]
    s["dev"] = tuple(torch.from_numpy(x).cuda() for x in (table, s["lens"], cu))
    return s


def expected(s, k_rows, v_rows):
    """The caches with the rows' codes and scale bytes at their tokens' slots, everything else as it is."""
    row, page, slot, _, _ = (torch.from_numpy(a) for a in ref.token_places(s["cu"], s["lens"], s["page"], s["table"]))
    out = [x.cpu().clone() for x in s["caches"]]
    for i, x in enumerate((k_rows, v_rows)):
        for to, put in zip((out[i], out[2 + i]), fp8_ref.quantise(x.cpu()[row], s["dtype"])):
            (to if s["order"] == "nhd" else to.transpose(1, 2))[page, slot] = put
    return out


def append(s, **kw):
    return sdpa.sdpa_paged_append_fp8(s["k"], s["v"], *s["caches"], *s["dev"], cache_layout=s["order"], **kw)


WRITES = [([1] * 5, [1, 17, 16, 33, 1000]), ([0, 3, 0, 70, 1], [0, 3, 40, 129, 64]), ([1], [1]), ([257], [257]),
          ([2] * 70, list(range(2, 72)))]


@pytest.mark.parametrize("new,total", WRITES)
@pytest.mark.parametrize("d,dv,page,order", [(128, 128, 16, "nhd"), (256, 256, 48, "hnd"), (192, 128, 32, "hnd"),
                                             (512, 512, 256, "nhd")])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_copied_rows(new, total, d, dv, page, order, dtype):
    s = write_batch(1, new, total, page, 3, d, dv, order, dtype, pad=4, std=3.0)
    want = expected(s, s["k"], s["v"])
    assert append(s) is None and sdpa.sdpa_last_launch_count() == 1
    assert all(torch.equal(a.cpu(), b) for a, b in zip(s["caches"], want))
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [128, 192, 256, 512])
def test_rows_at_the_borders(dtype, d):
    """Zeros, one value, largest magnitudes at and next to the borders of the exponent, at the type's ends, subnormals,
    infinities, NaN."""
    info = torch.finfo(dtype)
    tops = [0.0, info.max, info.tiny, info.smallest_normal, 448.0, 450.0, 449.0, 224.0, 225.0, 1.75, 1.7578125, 1.0, 57344.0,
            2.0 ** -24, 2.0 ** -25 if dtype == BF else 2.0 ** -24, float("inf")]
    tops += [2.0 ** x for x in ((-120, -100, -90, -88, -72, 60, 88, 90, 100) if dtype == BF else (-14, -10, -7, 8, 14, 15))]
    g = torch.Generator().manual_seed(3)
    x = (torch.rand(len(tops) * 2, 1, d, generator=g) * 2 - 1).double()
    for i, t in enumerate(tops):
        for j in (2 * i, 2 * i + 1):
            x[j] *= min(t, float(info.max))
            x[j, 0, j * 5 % d] = t if j % 2 else -t
    x = x.to(dtype)
    x[1, 0, 7], x[4, 0, 0], x[9, 0, d - 1] = float("nan"), float("nan"), float("-inf")
    n = x.shape[0]
    s = write_batch(5, [n], [n + 3], 16, 1, d, 128 if d == 192 else d, "nhd", dtype)
    s["k"] = x.cuda()
    s["v"] = x.flip(0)[..., :s["v"].shape[-1]].contiguous().cuda()
    want = expected(s, s["k"], s["v"])
    append(s)
    for a, b in zip(s["caches"], want):
        a = a.cpu()
        same = (a == b) | ((a & 127) == 127) & ((b & 127) == 127)  # a NaN's sign is free
        assert bool(same.all())


@pytest.mark.parametrize("d,dv,rot,inter,sections", [(128, 128, 128, False, None), (192, 128, 64, False, (16, 10, 6)),
                                                     (256, 256, 256, True, (42, 43, 43)), (512, 512, 128, False, None),
                                                     (128, 128, 0, False, None), (128, 128, 128, True, (22, 21, 21))])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_normed_rotated_and_quantised(d, dv, rot, inter, sections, dtype):
    s = write_batch(2, [0, 3, 0, 70, 1], [0, 3, 40, 129, 64], 16, 2, d, dv, "nhd", dtype, pad=3, hq=6)
    g = torch.Generator().manual_seed(8)
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=g)).to(dtype)
    table = ref.angles_table(1000, rot)
    row, page, slot, pos, _ = (torch.from_numpy(a) for a in ref.token_places(s["cu"], s["lens"], 16, s["table"]))
    rows = s["k"].shape[0]
    axes = 1 if sections is None else len(sections)
    where = torch.zeros(axes, rows, dtype=torch.int32)
    for a in range(axes):
        where[a, row] = ((pos * (1 + 6 * a) + 3 * a) % 1000).int()
    positions = None if rot == 0 or sections is None else where.cuda()
    before = [x.cpu().clone() for x in s["caches"]]
    v_want = expected(s, s["k"], s["v"])
    q_out = torch.full_like(s["q"].contiguous(), 5.0)
    got = append(s, q=s["q"], q_weight=wq.cuda(), k_weight=wk.cuda(), cos_sin=None if table is None else table.cuda(),
                 positions=positions, interleaved=inter, sections=sections, q_out=q_out)
    assert got is q_out and sdpa.sdpa_get_device_error() == 0
    # q as the norm and rotation alone give it
    at = None if rot == 0 else (where if sections is not None else where[0]).cuda()
    q_ref, _ = sdpa.sdpa_qk_norm_rope(s["q"], s["k"], wq.cuda(), wk.cuda(), None if table is None else table.cuda(), at,
                                      interleaved=inter, sections=sections)
    assert torch.equal(q_out[:-3], q_ref[:-3]) and bool((q_out[-3:] == 5).all())
    after = [x.cpu() for x in s["caches"]]
    assert torch.equal(after[1], v_want[1]) and torch.equal(after[3], v_want[3])
    if rot == 0:
        angles = None
    elif sections is None:
        angles = table[where[0].long()]
    else:
        from test_gpu_rope_axes import merged

        angles = merged(table, where, sections)
    y, mag = ref.norm_rope(s["k"].cpu(), wk, angles, rot, 1e-6, inter)
    y, mag = y[row], mag[row]
    e = after[2][page, slot].long() - 127
    exact = torch.from_numpy(fp8_ref.exponent(y.abs().amax(-1).numpy(), dtype))
    top = y.abs().amax(-1)
    border = (top / (448 * torch.exp2(exact.double())) - 1).abs().minimum((top / (224 * torch.exp2(exact.double())) - 1).abs())
    assert bool(((e == exact) | (((e - exact).abs() == 1) & (border < 2.0 ** -18))).all())
    stored = fp8_ref.decode(after[0][page, slot], after[2][page, slot])
    tol = (2.0 ** -4 * y.abs() + 2.0 ** -10 * torch.exp2(e.double())[..., None]) + 2.0 ** -18 * mag
    assert bool(((stored - y).abs() <= tol).all())
    # everything but the new tokens' slots as it was
    for a, b in ((after[0], before[0]), (after[2], before[2])):
        a[page, slot] = 0
        b[page, slot] = 0
        assert torch.equal(a, b)


def test_skipped_tokens():
    """Bad lengths and pages leave their tokens out and the rest in."""
    for what, code in (("len", 6), ("page", 10)):
        s = write_batch(4, [2, 1, 3], [20, 30, 40], 16, 2, 128, 128, "nhd", BF)
        want = expected(s, s["k"], s["v"])
        clean = [x.cpu().clone() for x in s["caches"]]
        table, lens, cu = (x.clone() for x in s["dev"])
        if what == "len":
            lens[1] = 0
        else:
            table[1, 1] = -5
        s["dev"] = (table, lens, cu)
        append(s)
        assert sdpa.sdpa_get_device_error() == code
        p, slot = int(s["table"][1, 29 // 16]), 29 % 16
        for a, b, c in zip(s["caches"], want, clean):
            b[p, slot] = c[p, slot]
            assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("order", ["nhd", "hnd"])
def test_blocks_of_codes_and_scales(order):
    """A page's K, V and scale bytes in one block, written, read and attended through slices of it."""
    d, page, hkv, new, total = 128, 16, 2, [1, 4, 2], [50, 4, 33]
    s = write_batch(6, new, total, page, hkv, d, d, order, BF)
    pages = s["caches"][0].shape[0]
    n = page * hkv
    # a page's stride is a multiple of its slots' and heads' (a copy's rule): the block ends in padding
    block = torch.zeros(pages, 2 * n * d + -(-2 * n // (hkv * page * d)) * hkv * page * d, dtype=torch.uint8, device="cuda")
    heads = (page, hkv) if order == "nhd" else (hkv, page)
    kc, vc = (block[:, x * n * d:(x + 1) * n * d].view(pages, *heads, d) for x in (0, 1))
    ks, vs = (block[:, 2 * n * d + x * n:2 * n * d + (x + 1) * n].view(pages, *heads) for x in (0, 1))
    for a, b in zip((kc, vc, ks, vs), s["caches"]):
        a.copy_(b)
    want = expected(s, s["k"], s["v"])
    s["caches"] = [kc, vc, ks, vs]
    append(s)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(s["caches"], want))
    # filled whole, then read and attended
    for x, y in zip(s["caches"][:2], s["caches"][2:]):
        codes, scale = fp8_ref.quantise(torch.randn(x.shape), BF)
        x.copy_(codes), y.copy_(scale)
    copies = [x.contiguous() for x in s["caches"]]
    cu = torch.tensor([0, 50, 54, 87], dtype=torch.int32, device="cuda")
    a = sdpa.sdpa_paged_read_fp8(*s["caches"], s["dev"][0], s["dev"][1], cu, cache_layout=order, rows=87, dtype=BF)
    b = sdpa.sdpa_paged_read_fp8(*copies, s["dev"][0], s["dev"][1], cu, cache_layout=order, rows=87, dtype=BF)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q = torch.randn(7, 6, d, device="cuda").bfloat16()
    a, b = (sdpa.sdpa_paged_fwd_fp8(q, *x, *s["dev"], max_seqlen_q=4, cache_layout=order) for x in (s["caches"], copies))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and sdpa.sdpa_get_device_error() == 0


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("take,total", [([5, 0, 17, 300, 1], [5, 40, 30, 300, 1000]), ([1], [1]), ([1000], [1000]),
                                        ([2] * 70, list(range(2, 72)))])
@pytest.mark.parametrize("d,page,order", DIMS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_read(take, total, d, page, order, dtype):
    c = case([1] * len(total), total, hkv=3, hq=3, d=d, page=page, order=order, dtype=dtype, seed=2)
    cu = np.concatenate([[0], np.cumsum(take)]).astype(np.int32)
    rows = int(cu[-1]) + 2
    dv = c["vc"].shape[-1]
    wide = torch.full((rows, 3 * (d + dv) + 8), 7.0, dtype=dtype, device="cuda")
    k_out = wide[:, :3 * d].unflatten(1, (3, d))
    v_out = wide[:, 3 * d:3 * (d + dv)].unflatten(1, (3, dv))
    got = sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], torch.from_numpy(cu).cuda(), cache_layout=order, k_out=k_out, v_out=v_out)
    assert got[0] is k_out and got[1] is v_out and sdpa.sdpa_last_launch_count() == 1
    row, pg, slot, _, _ = (torch.from_numpy(a) for a in ref.token_places(cu, c["lens"], page, c["table"]))
    for out, x in ((k_out.cpu(), c["kc"]), (v_out.cpu(), c["vc"])):
        assert torch.equal(out[row].double(), x[pg, slot])  # exact in the type
        assert bool((out[int(cu[-1]):] == 7).all())
    assert bool((wide[:, 3 * (d + dv):] == 7).all()) and sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("take", [[3333, 0, 1, 3403], [3300, 3303], [1] * 7 + [12793]])
@pytest.mark.parametrize("hkv,d,order", [(1, 128, "nhd"), (2, 192, "hnd"), (1, 512, "nhd"), (4, 128, "nhd"), (5, 128, "nhd")])
def test_read_of_many_rows_of_few_heads(take, hkv, d, order):
    """Rows enough that a warp walks several tokens of few heads at once; its last ones end behind the batch."""
    total = [t + 5 for t in take]
    c = case([1] * len(total), total, hkv=hkv, hq=hkv, d=d, order=order, seed=4)
    cu = np.concatenate([[0], np.cumsum(take)]).astype(np.int32)
    n = int(cu[-1])
    row, pg, slot, _, _ = (torch.from_numpy(a) for a in ref.token_places(cu, c["lens"], c["page"], c["table"]))
    table = c["dev"][5].clone()
    bad = max(range(len(take)), key=lambda b: take[b])
    table[bad, 20] = -1
    gone = (pg == int(c["table"][bad, 20]))
    k, v = sdpa.sdpa_paged_read_fp8(*c["dev"][1:5], table, c["dev"][6], torch.from_numpy(cu).cuda(), cache_layout=order,
                                    k_out=torch.full((n + 3, hkv, d), 7.0, dtype=BF, device="cuda"),
                                    v_out=torch.full((n + 3, hkv, c["vc"].shape[-1]), 7.0, dtype=BF, device="cuda"))
    assert sdpa.sdpa_get_device_error() == 10 and int(gone.sum()) == 16
    for out, x in ((k.cpu(), c["kc"]), (v.cpu(), c["vc"])):
        assert torch.equal(out[row[~gone]].double(), x[pg[~gone], slot[~gone]])
        assert bool((out[row[gone]] == 7).all()) and bool((out[n:] == 7).all())


def test_read_special_codes_and_other_types():
    """Every code with scales from one end to the other, rounded once into the other type too."""
    scales = [0, 1, 20, 47, 60, 112, 118, 126, 127, 128, 134, 150, 207, 230, 254, 255]
    kc = torch.arange(256, dtype=torch.uint8).view(1, 1, 2, 128).expand(1, 16, 2, 128).contiguous()
    ks = torch.tensor(scales, dtype=torch.uint8).view(1, 16, 1).expand(1, 16, 2).contiguous()
    table, lens = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([16], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 16], dtype=torch.int32).cuda()
    for dtype in (BF, HF):
        k, v = sdpa.sdpa_paged_read_fp8(kc.cuda(), kc.cuda(), ks.cuda(), ks.cuda(), table, lens, cu, rows=16, dtype=dtype)
        assert torch.equal(torch.nan_to_num(k), torch.nan_to_num(v))
        s = torch.exp2(ks[0].double() - 127)
        s = torch.where(ks[0] == 0, 0.0, torch.where(ks[0] == 255, float("inf"), s))
        want = (torch.from_numpy(fp8_ref.VALUES)[kc[0].long()] * s[..., None]).float().to(dtype)
        same = (k.cpu() == want) | (torch.isnan(k.cpu()) & torch.isnan(want))
        assert bool(same.all())


def test_read_skips_what_is_bad():
    c = case([1] * 3, [20, 30, 40], hkv=2, hq=2, d=128)
    cu = torch.tensor([0, 20, 50, 90], dtype=torch.int32, device="cuda")
    good = sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], cu, rows=90, dtype=BF)
    for what, code in (("len", 6), ("page", 10)):
        table, lens = c["dev"][5].clone(), c["dev"][6].clone()
        if what == "len":
            lens[1] = 12  # 30 rows asked for
        else:
            table[1, 1] = 1 << 20
        k, v = (torch.full_like(x, 3.0) for x in good)
        sdpa.sdpa_paged_read_fp8(*c["dev"][1:5], table, lens, cu, k_out=k, v_out=v)
        assert sdpa.sdpa_get_device_error() == code
        for a, b in ((k, good[0]), (v, good[1])):
            assert torch.equal(a[:20], b[:20]) and torch.equal(a[50:], b[50:])
            skipped = slice(20, 38) if what == "len" else slice(36, 50)
            assert bool((a[skipped] == 3).all())


# ---------------------------------------------------------------- a run of them

@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (256, 4, 2)])
def test_prompt_then_decoding(d, hq, hkv):
    """A prompt in two chunks and five decoding steps: each step's append, then attention over the cache; a chunk's
    attention also from the rows read back through sdpa_fwd, which sees the same values."""
    g = torch.Generator(device="cuda").manual_seed(1)
    batch, page, sections = 3, 16, (16, 24, 24)
    wq, wk = (1 + 0.2 * torch.randn(2, d, device="cuda", generator=g)).bfloat16()
    table = ref.angles_table(400, 128).cuda()
    pages = 3 * 12
    kc, vc = (torch.zeros(pages, page, hkv, d, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(pages, page, hkv, dtype=torch.uint8, device="cuda") for _ in "kv")
    ids = torch.randperm(pages, device="cuda", generator=g).int().view(3, 12).contiguous()
    have = np.zeros(batch, dtype=np.int64)
    for new in ([40, 75, 3], [60, 0, 50]) + ([1, 1, 1],) * 5:
        have += new
        rows = int(sum(new))
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        lens = torch.from_numpy(have.astype(np.int32)).cuda()
        x = torch.randn(rows, (hq + 2 * hkv) * d, device="cuda", generator=g).bfloat16()
        q, k, v = x.split([hq * d, hkv * d, hkv * d], dim=1)
        q, k, v = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
        pos = torch.randint(0, 400, (3, rows), device="cuda", generator=g, dtype=torch.int32)
        q_rot = sdpa.sdpa_paged_append_fp8(k, v, kc, vc, ks, vs, ids, lens, cu, q=q, q_weight=wq, k_weight=wk, cos_sin=table,
                                           positions=pos, sections=sections)
        o, lse = sdpa.sdpa_paged_fwd_fp8(q_rot, kc, vc, ks, vs, ids, lens, cu, max_seqlen_q=max(new))
        cu_k = torch.from_numpy(np.concatenate([[0], np.cumsum(have)]).astype(np.int32)).cuda()
        kr, vr = sdpa.sdpa_paged_read_fp8(kc, vc, ks, vs, ids, lens, cu_k, rows=int(have.sum()), dtype=BF)
        c = dict(q=q_rot.cpu(), kc=fp8_ref.decode(kc.cpu(), ks.cpu()), vc=fp8_ref.decode(vc.cpu(), vs.cpu()), table=ids.cpu().numpy(),
                 cu=cu.cpu().numpy(), lens=have.astype(np.int32), page=page, max_kv=int(have.max()), scale=d ** -0.5, dtype=BF)
        check(c, o, lse)
        if min(new) > 0:
            o2, lse2 = sdpa.sdpa_fwd(q_rot, kr, vr, layout="thd", mask="causal_br", cu_seqlens_q=cu, cu_seqlens_kv=cu_k,
                                     max_seqlen_q=max(new), max_seqlen_kv=int(have.max()))
            # two kernels within their tolerances of the same result: P to 2^-8 and 2^-10, O to 2^-8 each
            _, _, pv, _ = ref.paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], page, "nhd", True, -1, c["scale"])
            assert bool(((o - o2).cpu().double().abs() <= (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -7 + 2.0 ** -10) * pv + 1e-6).all())
            assert bool(((lse - lse2).abs() <= 2.0 ** -15 * (1 + lse.abs())).all())


# ---------------------------------------------------------------- how a program calls them

def test_many_tiles_and_many_items():
    """Rings go round many times, items cross many cuts, every tile of a short item is an edge."""
    for new, total, d, kw in (([1] * 40, [1 + 97 * i for i in range(40)], 128, {}), ([3] * 200, [3 + i % 61 for i in range(200)], 256, {}),
                              ([2] * 12, [5000] * 12, 512, {}), ([64], [3000], 128, {}), ([100, 1], [4000, 9000], 192, {})):
        c = case(new, total, d=d, page=16, **kw)
        c["vmax"] = used_vmax(c)
        check(c, *call(c))
        check(c, *call(c, window=200), window=200)


def test_a_large_batch():
    n = 700
    c = case([i % 3 for i in range(n)], [max(i % 3, (i * 37) % 400) for i in range(n)], hq=4, hkv=1, d=128)
    c["vmax"] = used_vmax(c)
    check(c, *call(c))


def test_strided_queries_and_a_wide_table():
    """q rows in a wider projection, not a multiple of head_dim apart; a block table that is a slice of a wider one."""
    for d in (128, 192):
        c = case([2, 1, 4], [130, 300, 77], d=d, page=32)
        wide = torch.full((7, 8 * d + 24), float("nan"), dtype=BF, device="cuda")
        wide[:, 8:8 + 8 * d] = c["dev"][0].reshape(7, -1)
        table = torch.full((3, c["dev"][5].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
        table[:, 2:-3] = c["dev"][5]
        want = call(c)
        c["dev"][0], c["dev"][5] = wide[:, 8:8 + 8 * d].unflatten(1, (8, d)), table[:, 2:-3]
        got = call(c)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        c["vmax"] = used_vmax(c)
        check(c, *got)


def test_offsets_beyond_32_bits():
    """Pages whose codes lie more than 4 GiB into the cache: written, read back and attended."""
    d, page, hkv, pages = 128, 16, 8, 270000
    kc, vc = (torch.empty(pages, page, hkv, d, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.empty(pages, page, hkv, dtype=torch.uint8, device="cuda") for _ in "kv")
    assert kc.numel() > 2 ** 32
    ids = torch.tensor([[269999, 3, 265000, 131072, 262145]], dtype=torch.int32, device="cuda")
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([75], [0, 75]))
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(75, hkv, d, device="cuda", generator=g).bfloat16() for _ in "kv")
    sdpa.sdpa_paged_append_fp8(k, v, kc, vc, ks, vs, ids, lens, cu)
    kr, vr = sdpa.sdpa_paged_read_fp8(kc, vc, ks, vs, ids, lens, cu, rows=75, dtype=BF)
    for x, y in ((k, kr), (v, vr)):
        assert torch.equal(y.cpu().double(), fp8_ref.decode(*fp8_ref.quantise(x.cpu(), BF)))
    q = torch.randn(3, 8, d, device="cuda", generator=g).bfloat16()
    small = [x[ids[0].long()].contiguous() for x in (kc, vc, ks, vs)]
    near = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    cu3 = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    a = sdpa.sdpa_paged_fwd_fp8(q, kc, vc, ks, vs, ids, lens, cu3, max_seqlen_q=3)
    b = sdpa.sdpa_paged_fwd_fp8(q, *small, near, lens, cu3, max_seqlen_q=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and sdpa.sdpa_get_device_error() == 0


def test_two_calls_at_once_on_two_streams():
    c, e = case([6, 1, 5], [900, 2000, 300], pad=1), case([1, 3, 20], [1500, 700, 800], d=256, page=64, order="hnd")
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [(call(c, stream=streams[0]), call(e, stream=streams[1])) for _ in range(10)]
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[0][:-1], got[0][0][0][:-1]) and torch.equal(b[0], got[0][1][0])
    for x, y in ((c, got[-1][0]), (e, got[-1][1])):
        x["vmax"] = used_vmax(x)
        check(x, *y)
    # append and read on a stream of their own
    s = write_batch(1, [3, 0, 70], [3, 40, 129], 16, 2, 128, 128, "nhd", BF)
    want = expected(s, s["k"], s["v"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    append(s, stream=side)
    kr, vr = sdpa.sdpa_paged_read_fp8(*s["caches"], *s["dev"], rows=73, dtype=BF, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(s["caches"], want))
    assert torch.equal(kr.cpu().double(), fp8_ref.decode(*fp8_ref.quantise(s["k"].cpu(), BF)))


def test_captured_steps_follow_the_lengths_and_share_a_workspace():
    """Two captured graphs, an append with attention each, that use one workspace in turn; lengths, tables and tokens
    change in place between replays."""
    d, hq, hkv, page, batch = 128, 8, 2, 16, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    caches = [torch.zeros(40, page, hkv, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    caches += [torch.full((40, page, hkv), 127, dtype=torch.uint8, device="cuda") for _ in "kv"]
    ids = torch.arange(40, dtype=torch.int32, device="cuda").view(batch, 10).contiguous()
    lens, cu = torch.ones(batch, dtype=torch.int32, device="cuda"), torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    x = torch.randn(batch, (hq + 2 * hkv) * d, device="cuda", generator=g).bfloat16()
    q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([hq * d, hkv * d, hkv * d], dim=1))
    ws = torch.empty(sdpa.PAGED_WORKSPACE_MAX, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for bound in (160, 64):
        o, lse = torch.zeros(batch, hq, d, dtype=BF, device="cuda"), torch.zeros(batch, hq, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sdpa.sdpa_paged_append_fp8(k, v, *caches, ids, lens, cu)
            sdpa.sdpa_paged_fwd_fp8(q, *caches, ids, lens, cu, max_seqlen_q=1, max_seqlen_kv=bound, out=o, lse=lse, workspace=ws)
        outs.append((o, lse))
        graphs.append(graph)
    for step in range(12):
        n = [1 + step, 1 + 2 * step, 1 + 3 * step, 1 + 4 * step]
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        for graph in graphs:
            graph.replay()
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        c = dict(q=q.cpu(), kc=fp8_ref.decode(caches[0].cpu(), caches[2].cpu()), vc=fp8_ref.decode(caches[1].cpu(), caches[3].cpu()),
                 table=ids.cpu().numpy(), cu=cu.cpu().numpy(), lens=np.array(n, dtype=np.int32), page=page, max_kv=max(n),
                 scale=d ** -0.5, dtype=BF)
        check(c, *outs[0])


@pytest.mark.parametrize("name,d", [("ragged", 128), ("spec", 192), ("chunk", 256), ("spec", 512)])
def test_a_workspace_of_the_reported_size_is_enough(name, d, monkeypatch):
    c = case(*BATCHES[name], d=d)
    c["vmax"] = used_vmax(c)
    sizes, launch = [], sdpa._launch
    monkeypatch.setattr(sdpa, "_launch", lambda n, dev, *a: (sizes.append(a[-1]), launch(n, dev, *a)))
    call(c)
    guard = torch.full((sizes[0] + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = call(c, workspace=guard[:sizes[0]])
    check(c, o, lse)
    assert bool((guard[sizes[0]:] == 0xA5).all())


@pytest.mark.parametrize("d,order", [(128, "nhd"), (192, "hnd"), (256, "hnd"), (512, "nhd")])
def test_every_access_is_inside_the_buffers(d, order):
    """The address-checked build: attention, append (copied; normed, with axes) and read, the same bits as the other one."""
    for name in ("ragged", "spec", "chunk", "short_cache"):
        c = case(*BATCHES[name], d=d, order=order, page=48)
        want = call(c)
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(c["lens"])]).astype(np.int32)).cuda()
        rows = int(c["lens"].sum())
        back = sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], cu, cache_layout=order, rows=rows, dtype=BF)
        s = write_batch(3, *WRITES[1], 16, 2, d, 128 if d == 192 else d, order, BF, pad=3, hq=4)
        w = torch.ones(d, device="cuda").bfloat16()
        t, pos = ref.angles_table(100, 48).cuda(), torch.randint(0, 100, (2, s["k"].shape[0]), device="cuda", dtype=torch.int32)
        norm = dict(q=s["q"], q_weight=w, k_weight=w, cos_sin=t, positions=pos, sections=(11, 13))
        clean = [x.clone() for x in s["caches"]]
        append(s), append(s, **norm)
        written = [x.clone() for x in s["caches"]]
        both = sdpa.sdpa_qk_norm_rope(s["q"], s["k"], w, w, t, pos, sections=(11, 13))
        with sdpa.address_checked():
            sdpa.sdpa_debug_address_report()
            got = call(c)
            again = sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], cu, cache_layout=order, rows=rows, dtype=BF)
            for x, y in zip(s["caches"], clean):
                x.copy_(y)
            append(s), append(s, **norm)
            rope = sdpa.sdpa_qk_norm_rope(s["q"], s["k"], w, w, t, pos, sections=(11, 13))
            assert sdpa.sdpa_debug_address_report()[0] == 0 and sdpa.sdpa_get_device_error() == 0
        for a, b in zip(got + again + rope + tuple(s["caches"]), want + back + both + tuple(written)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("hkv,d,n", [(1, 128, 4005), (2, 192, 8201), (1, 512, 13001), (8, 128, 40100)])
def test_long_reads_stay_inside_the_buffers(hkv, d, n):
    """The read's forms for many rows: their outputs and scales end where the last row does."""
    c = case([1, 1], [n - 3, 3], hkv=hkv, hq=hkv, d=d, seed=6, poison=False)
    cu = torch.tensor([0, n - 3, n], dtype=torch.int32, device="cuda")
    want = sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], cu, rows=n, dtype=BF)
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        got = sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], cu, rows=n, dtype=BF)
        assert sdpa.sdpa_debug_address_report()[0] == 0 and sdpa.sdpa_get_device_error() == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_the_checker_sees_the_new_accesses():
    """With every extent 16 bytes short the last bytes of the scales and outputs count as outside, and are not written."""
    c = case([1, 1], [16, 32], hq=2, hkv=2, d=128)
    want = call(c)
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        try:
            sdpa.sdpa_debug_address_shrink(16)
            out = torch.full_like(want[0], 7.0)
            call(c, out=out)
            assert sdpa.sdpa_debug_address_report()[0] > 0 and sdpa.sdpa_get_device_error() == 9
        finally:
            sdpa.sdpa_debug_address_shrink(0)
        assert bool((out.flatten()[-8:] == 7).all())


def test_kernel_kinds_are_timed():
    c = case([1, 2], [300, 40])
    cu = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    sdpa.sdpa_profile_begin()
    call(c)
    sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], cu, rows=3, dtype=BF)
    got = sdpa.sdpa_profile_end()
    assert got["paged"][1] == 1 and got["read"][1] == 1 and got["paged"][0] > 0 and got["read"][0] > 0


def test_attention_of_a_long_chunk_agrees_with_rows_read_back():
    """300 tokens over 1000 keys: the kernel for few tokens in many items, and sdpa_fwd over the rows read back."""
    c = case([300], [1000], hq=8, hkv=2, d=128)
    c["vmax"] = used_vmax(c)
    o, lse = call(c)
    check(c, o, lse)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (300, 1000))
    k, v = sdpa.sdpa_paged_read_fp8(*c["dev"][1:7], cu_k, rows=1000, dtype=BF)
    o2, lse2 = sdpa.sdpa_fwd(c["dev"][0], k, v, layout="thd", mask="causal_br", cu_seqlens_q=cu_q, cu_seqlens_kv=cu_k,
                             max_seqlen_q=300, max_seqlen_kv=1000)
    _, _, pv, _ = ref.paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], 16, "nhd", True, -1, c["scale"])
    assert bool(((o - o2).cpu().double().abs() <= (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -7 + 2.0 ** -10) * pv + 1e-6).all())
    assert bool(((lse - lse2).abs() <= 2.0 ** -15 * (1 + lse.abs())).all())


@pytest.mark.parametrize("d", [128, 256, 512])
def test_cuts_anywhere(d):
    """Every number of CTAs up to 48: shares begin and end at every place of an item, also where it has no tiles yet."""
    c = case([1, 2, 1, 0, 1], [700, 530, 1, 40, 1025], hq=4, hkv=2, d=d, page=32)
    c["vmax"] = used_vmax(c)
    try:
        for cap in range(1, 49):
            sdpa.sdpa_debug_set_max_ctas(cap)
            check(c, *call(c))
    finally:
        sdpa.sdpa_debug_set_max_ctas(0)


def test_not_finite_across_cuts():
    """A query that is not finite stays NaN where its keys are divided between CTAs, whose parts are joined."""
    c = case([1, 1], [6000, 3000], hq=4, hkv=2, d=128)
    good, good_l = call(c)
    c["dev"][0] = c["dev"][0].clone()
    c["dev"][0][0, 1, 5], c["dev"][0][1, 2, 7] = float("-inf"), float("nan")
    o, lse = call(c)
    bad = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    assert bool(torch.isnan(o[bad]).all()) and not bool(torch.isfinite(lse[bad]).any())
    assert torch.equal(o[~bad], good[~bad]) and torch.equal(lse[~bad], good_l[~bad])
