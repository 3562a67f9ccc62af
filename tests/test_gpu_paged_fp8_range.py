"""Attention over the 8-bit paged cache at the ends of its numbers: value rows that
lie up to 2^160 apart, rows of zeros beside the largest, against the definition in
64 bits.

Tolerances, before the first run. Beside test_gpu_paged_fp8.py's terms: what a weight
P 2^ev loses in its three 8-bit terms is a step relative to itself and 2^-28 of the
largest weight that its row has (2^-17, half of the last term's least step, over
2^11, the least that the largest one is held as). A key's value is at most 448 2^ev, so n keys lose
at most n 2^-28 448 max_j p_j 2^ev_j, with p the row's own probabilities.
  |O - O'| <= (2^-10 + 2 s_err + 2^-19) sum p|v| + u |O| + n 2^-28 448 max_j p_j 2^ev_j
  |LSE - LSE'| <= s_err + 2^-19 (1 + |LSE|),   s_err = 2.5 (D/8) 2^-23 sum |q||k| scale
Denominators have no part in the values' exponents, so nothing in the LSE depends on them.
"""
import numpy as np
import pytest
import torch

import fp8_ref
import paged_ref as ref
import scaled_dot_product_02_gb300 as sdpa
from test_gpu_paged_fp8 import call, case

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def places(c, b):
    p = np.arange(c["lens"][b])
    return torch.from_numpy(c["table"][b, p // c["page"]].astype(np.int64)), torch.from_numpy(p % c["page"])


def rewrite(c, which, rows):
    """The keys' rows of "k" or "v" replaced: rows(b) is [lens[b], heads, width] of sequence b, any type."""
    name, at, s_at = ("kc", 1, 3) if which == "k" else ("vc", 2, 4)
    codes, scale = c["dev"][at].cpu(), c["dev"][s_at].cpu()
    if c["order"] == "hnd":
        codes, scale = codes.transpose(1, 2).contiguous(), scale.transpose(1, 2).contiguous()
    for b in range(len(c["lens"])):
        where = places(c, b)
        codes[where], scale[where] = fp8_ref.quantise(rows(b), c["dtype"])
    c[name] = fp8_ref.decode(codes, scale)
    for i, x in ((at, codes), (s_at, scale)):
        c["dev"][i] = (x if c["order"] == "nhd" else x.transpose(1, 2).contiguous()).cuda()


def largest_weight(c):
    """max_j p_j 2^ev_j of every row and head, [rows, heads] float64 (causal)."""
    scale = c["dev"][4].cpu()
    scale = scale if c["order"] == "nhd" else scale.transpose(1, 2)
    rows, hq, d = c["q"].shape
    g = hq // c["kc"].shape[2]
    out = torch.zeros(rows, hq, dtype=torch.float64)
    for b, n in enumerate(c["lens"]):
        lo, hi = int(c["cu"][b]), int(c["cu"][b + 1])
        if lo == hi or n == 0:
            continue
        where = places(c, b)
        k, by = c["kc"][where], torch.exp2(scale[where].double() - 127)
        hidden = torch.arange(int(n))[None, :] > torch.arange(int(n) - (hi - lo), int(n))[:, None]
        for h in range(hq):
            s = c["q"][lo:hi, h].double() @ k[:, h // g].T * c["scale"]
            s[hidden] = -np.inf
            out[lo:hi, h] = (torch.softmax(s, -1) * by[:, h // g]).amax(-1)
    return out


def tolerances(c):
    d, live = c["q"].shape[-1], int(c["cu"][-1])
    want, want_l, pv, mag = ref.paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], c["page"], "nhd",
                                                True, -1, c["scale"])
    want, want_l, pv, mag = (x[:live] for x in (want, want_l, pv, mag))
    s_err = 2.5 * (d / 8) * 2.0 ** -23 * mag
    floor = int(max(c["lens"])) * 2.0 ** -28 * 448 * largest_weight(c)[:live]
    tol = (2.0 ** -10 + 2 * s_err + 2.0 ** -19)[..., None] * pv + ref.U[c["dtype"]] * want.abs() + ref.TINY[c["dtype"]]
    return want, want_l, tol + floor[..., None], s_err + 2.0 ** -19 * (1 + want_l.abs())


def check(c, o, lse, expected):
    want, want_l, tol, tol_l = expected
    o, lse = o[:len(want)].cpu().double(), lse[:len(want)].cpu().double()
    assert bool(torch.isfinite(lse).all())
    err = (lse - want_l).abs()
    assert bool((err <= tol_l).all()), f"LSE: worst {(err / tol_l).max().item():.2f} of the tolerance"
    err = (o - want).abs()
    assert bool((err <= tol).all()), f"O: worst {(err / tol).max().item():.2f} of the tolerance"
    assert sdpa.sdpa_get_device_error() == 0


PLACES = {  # which keys have the large values, the others zeros
    "within a tile": lambda p, n: p % 2 == 0,
    "tiles in turn": lambda p, n: p // 128 % 2 == 0,
    "the other tiles": lambda p, n: p // 128 % 2 == 1,
    "second half": lambda p, n: p >= n // 2,
    "first half": lambda p, n: p < n // 2,
    "the last key": lambda p, n: p == n - 1,
    "the first key": lambda p, n: p == 0,
}


@pytest.mark.parametrize("where", PLACES)
@pytest.mark.parametrize("d,hq,hkv,order", [(128, 4, 1, "nhd"), (192, 32, 2, "hnd"), (256, 8, 2, "nhd"), (512, 8, 1, "hnd")])
def test_rows_of_zeros_beside_the_largest(d, hq, hkv, order, where):
    """A zero row has the least scale byte; its key's share of the sum is that of any other."""
    for e in (50, 70, 87):
        c = case([1, 5], [1300, 700], hq=hq, hkv=hkv, d=d, order=order, seed=e)
        g = torch.Generator().manual_seed(e)

        def rows(b):
            n = int(c["lens"][b])
            x = torch.randn(n, hkv, 128 if d == 192 else d, generator=g).clamp(-1.9, 1.9).double() * 2.0 ** e
            x[torch.from_numpy(~PLACES[where](np.arange(n), n))] = 0
            return x
        rewrite(c, "v", rows)
        expected = tolerances(c)
        try:
            for cap in (0, 1, 2, 7):  # whole items, and cuts at different keys
                sdpa.sdpa_debug_set_max_ctas(cap)
                check(c, *call(c), expected)
        finally:
            sdpa.sdpa_debug_set_max_ctas(0)


@pytest.mark.parametrize("kind", ["rising", "falling", "any"])
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 8), (192, 4, 1), (256, 16, 1), (512, 4, 2)])
def test_exponents_from_end_to_end(d, hq, hkv, kind):
    """Value rows with every exponent that there is, in order and without: the maximum moves with the values', what was
    summed before keeps its place."""
    c = case([2, 1, 9], [1500, 129, 640], hq=hq, hkv=hkv, d=d, seed=d)
    g, rng = torch.Generator().manual_seed(d), np.random.default_rng(d)

    def rows(b):
        n = int(c["lens"][b])
        e = {"rising": np.linspace(-88, 87, n), "falling": np.linspace(87, -88, n), "any": rng.uniform(-88, 87, n)}[kind]
        x = torch.randn(n, hkv, 128 if d == 192 else d, generator=g).clamp(-1.9, 1.9).double()
        return x * torch.exp2(torch.from_numpy(e))[:, None, None]
    rewrite(c, "v", rows)
    expected = tolerances(c)
    try:
        for cap in (0, 1, 5):
            sdpa.sdpa_debug_set_max_ctas(cap)
            check(c, *call(c), expected)
    finally:
        sdpa.sdpa_debug_set_max_ctas(0)


def test_fp16_rows_at_the_ends():
    c = case([1, 4], [900, 300], hq=8, hkv=2, d=128, dtype=HF)
    g = torch.Generator().manual_seed(1)

    def rows(b):
        x = torch.randn(int(c["lens"][b]), 2, 128, generator=g).clamp(-1.7, 1.7).half()
        x[::2] *= 2.0 ** 14
        x[1::4] = 0
        return x
    rewrite(c, "v", rows)
    check(c, *call(c), tolerances(c))


@pytest.mark.parametrize("spread", [2.0, 30.0, 80.0])
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 8), (256, 8, 2), (192, 32, 2), (512, 8, 2)])
def test_small_values_are_kept_beside_large_ones(d, hq, hkv, spread):
    """Tolerances by the row's own weights: zeros in place of a row's result are outside of them, whatever other rows hold."""
    for seed in range(2):
        c = case([1, 2, 1], [900, 513, 300], hq=hq, hkv=hkv, d=d, spread=spread, seed=seed)
        expected = tolerances(c)
        want, _, tol, _ = expected
        assert bool((tol.amax(-1) <= 2.0 ** -4 * want.abs().amax(-1)).all())
        assert bool(((tol < want.abs()).double().mean(-1) > 0.5).all())
        check(c, *call(c), expected)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (512, 2, 2)])
def test_scores_that_are_all_far_below_zero(d, hq, hkv):
    """Scores of -2^108 and below, one product each: the largest ones of a row share its weight, as any others would."""
    c = case([1, 3], [700, 200], hq=hq, hkv=hkv, d=d)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][..., 0] = 2.0 ** 110
    c["dev"][0] = c["q"].cuda()

    def rows(b):
        k = torch.zeros(int(c["lens"][b]), hkv, d)
        k[..., 0] = -torch.exp2(3.0 + torch.arange(int(c["lens"][b])) % 5)[:, None]
        return k
    rewrite(c, "k", rows)
    step = 2 * max(c["vc"][places(c, b)].abs().max().item() for b in range(2))  # above 448 2^ev: a row's largest code is over 224
    for cap in (0, 1, 5):
        sdpa.sdpa_debug_set_max_ctas(cap)
        try:
            o, lse = call(c)
        finally:
            sdpa.sdpa_debug_set_max_ctas(0)
        want_l = -2.0 ** 113 * c["scale"]  # the count's logarithm is far below a step
        assert bool(((lse.cpu().double() - want_l).abs() <= 2.0 ** -19 * abs(want_l)).all())
        for b, n in enumerate(c["lens"]):
            for i in range(int(c["cu"][b]), int(c["cu"][b + 1])):
                seen = int(n) - (int(c["cu"][b + 1]) - 1 - i)
                v = c["vc"][places(c, b)][:seen:5].repeat_interleave(hq // hkv, 1)
                want, pv = v.mean(0), v.abs().mean(0)
                tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -19) * pv + n * 2.0 ** -28 * step
                assert bool(((o[i].cpu().double() - want).abs() <= tol).all())
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (256, 4, 1)])
def test_queries_at_the_end_of_their_type(d, hq, hkv):
    """Queries whose products with codes pass fp32's largest number before the keys' scales make them small, or a scale of
    zero does; and the reverse."""
    c = case([1, 3], [700, 200], hq=hq, hkv=hkv, d=d)
    g = torch.Generator().manual_seed(9)
    k = [torch.randn(int(n), hkv, d, generator=g).double() for n in c["lens"]]
    for q_exp, k_exp, scale in ((120, -75, 2.0 ** -46), (100, 60, 0.0), (122, 2, 0.0), (-110, 80, 2.0 ** 29)):
        c["q"] = (torch.randn(4, hq, d, generator=g) * 2.0 ** q_exp).bfloat16()
        c["dev"][0], c["scale"] = c["q"].cuda(), scale
        rewrite(c, "k", lambda b: k[b] * 2.0 ** k_exp)
        check(c, *call(c), tolerances(c))


@pytest.mark.parametrize("dtype,top", [(BF, 2.0 ** 10), (BF, 2.0 ** 20), (BF, 2.0 ** 40), (HF, 2.0 ** 15)])
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (512, 8, 8)])
def test_a_channel_of_q_that_no_key_has(d, hq, hkv, dtype, top):
    """One value of a row outweighs all others and meets codes of zero. The others are held to half of the last term's least
    step, 2^-17, where the largest is brought to 2^14 or more: each is off by at most 2^-31 of it."""
    c = case([1, 3], [700, 200], hq=hq, hkv=hkv, d=d, dtype=dtype)
    c["q"][..., 7] = top
    c["dev"][0] = c["q"].cuda()
    g = torch.Generator().manual_seed(2)

    def rows(b):
        k = torch.randn(int(c["lens"][b]), hkv, d, generator=g)
        k[..., 7] = 0
        return k
    rewrite(c, "k", rows)
    largest = max(c["kc"][places(c, b)].abs().sum(-1).max().item() for b in range(2))
    extra = 2.0 ** -31 * top * largest * c["scale"]  # of a score
    want, want_l, tol, tol_l = tolerances(c)
    _, _, pv, _ = ref.paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["cu"], c["page"], "nhd", True, -1, c["scale"])
    o, lse = call(c)
    if extra < 0.1:  # a weight's and the sum's share: e^(2 x) - 1 <= 2.3 x
        check(c, o, lse, (want, want_l, tol + 2.3 * extra * pv, tol_l + extra))
    else:  # the scores say nothing any more: the mean of some values, and no more than that
        assert bool((o.cpu().double().abs() <= 1.01 * max(c["vc"][places(c, b)].abs().max().item() for b in range(2))).all())
        assert sdpa.sdpa_get_device_error() == 0
