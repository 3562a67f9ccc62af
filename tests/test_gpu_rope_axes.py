"""Norm + rotation with several positions a token, its gradient and the 16-bit
append, against the 64-bit reference of one position with the angles of every
pair taken from its axis's row. The arithmetic behind the angles is that of one
position, so the tolerances are test_gpu_norm_rope.py's, and equal positions on
all axes give its results bit for bit."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import scaled_dot_product_02_gb300 as sdpa
from test_gpu_norm_rope import EPS, check_forward, dev, make, within

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
MAX = 5000


def axes_positions(rows, axes, seed, max_pos=MAX):
    return torch.from_numpy(np.random.default_rng(seed + 77).integers(0, max_pos, (axes, rows)).astype(np.int32))


def merged(table, pos, sections):
    """The rows of angles that the tokens turn by, as one table [tokens, rot] to look up by token."""
    half, parts, at = table.shape[1] // 2, ([], []), 0
    for n, p in zip(sections, pos.long()):
        parts[0].append(table[p, at:at + n])
        parts[1].append(table[p, half + at:half + at + n])
        at += n
    return torch.cat(parts[0] + parts[1], dim=1)


# rows, hq, hkv, d, interleaved, fused, sections
CASES = [(1, 32, 8, 128, False, True, (16, 24, 24)), (77, 32, 8, 128, True, False, (22, 21, 21)),
         (5, 3, 1, 128, False, False, (1, 2, 5)), (300, 16, 4, 128, False, True, (1, 1, 1, 61)),
         (19, 14, 2, 192, False, True, (13, 17, 19, 47)), (33, 4, 4, 192, True, False, (48,)),
         (21, 16, 8, 256, False, False, (43, 43, 42)), (64, 16, 8, 256, True, True, (24, 20, 20)),
         (9, 2, 2, 256, False, False, (63, 65)), (13, 16, 4, 512, False, True, (86, 85, 85)),
         (40, 5, 5, 512, False, False, (35, 35, 34)), (2, 1, 1, 512, True, False, (253, 1, 1, 1))]


@pytest.mark.parametrize("rows,hq,hkv,d,inter,fused,sections", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward(rows, hq, hkv, d, inter, fused, sections, dtype):
    q, k, qd, kd, wq, wk, table, one = make(rows, hq, hkv, d, 2 * sum(sections), dtype, fused)
    pos = axes_positions(rows, len(sections), 1)
    call = lambda p, s: sdpa.sdpa_qk_norm_rope(qd, kd, dev(wq), dev(wk), dev(table), dev(p), eps=EPS,  # noqa: E731
                                               interleaved=inter, sections=s)
    qo, ko = call(pos, sections)
    assert sdpa.sdpa_last_launch_count() == 1
    angles, row = merged(table, pos, sections), torch.arange(rows)
    check_forward(qo, q, wq, angles, row, 2 * sum(sections), inter, dtype)
    check_forward(ko, k, wk, angles, row, 2 * sum(sections), inter, dtype)
    same = call(one.expand(len(sections), rows).contiguous(), sections)
    assert all(torch.equal(a, b) for a, b in zip(same, call(one, None)))
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("rows,hq,hkv,d,inter,fused,sections", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_backward(rows, hq, hkv, d, inter, fused, sections, dtype):
    rot = 2 * sum(sections)
    q, k, qd, kd, wq, wk, table, one = make(rows, hq, hkv, d, rot, dtype, fused)
    pos = axes_positions(rows, len(sections), 2)
    g = torch.Generator().manual_seed(9)
    gq, gk = torch.randn(q.shape, generator=g).to(dtype), torch.randn(k.shape, generator=g).to(dtype)
    call = lambda p, s: sdpa.sdpa_qk_norm_rope_bwd(dev(gq), dev(gk), qd, kd, dev(wq), dev(wk), dev(table), dev(p),  # noqa: E731
                                                   eps=EPS, interleaved=inter, sections=s)
    got, angles = call(pos, sections), merged(table, pos, sections)
    for x, w, dy, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        want, mag, want_w, mag_w = ref.norm_rope_bwd(dy, x, w, angles, rot, EPS, inter)
        within(dx, want, mag, ref.U[dtype], ref.TINY[dtype], 2.0 ** -17)
        within(dw, want_w, mag_w, 0.0, 0.0, 2.0 ** -15)
        # the slope of <dy, f(x + t v)> at 0 by central differences in 64 bits: off by t^2 / 6 of the third derivative
        # (t = 2^-13: below 1e-7 here) and by dx's own tolerance along v
        v = torch.randn(x.shape, generator=g, dtype=torch.float64)
        f = lambda t: (dy.double() * ref.norm_rope(x.double() + t * v, w, angles, rot, EPS, inter)[0]).sum()  # noqa: E731
        slope, t = (f(2.0 ** -13) - f(-2.0 ** -13)) * 2.0 ** 12, (dx.double().cpu() * v).sum()
        bound = ((ref.U[dtype] * want.abs() + ref.TINY[dtype] + 2.0 ** -17 * mag) * v.abs()).sum() + 1e-6 * (mag * v.abs()).sum()
        assert abs(float(slope - t)) <= float(bound)
    assert all(torch.equal(a, b) for a, b in zip(got, call(pos, sections)))
    same = call(one.expand(len(sections), rows).contiguous(), sections)
    assert all(torch.equal(a, b) for a, b in zip(same, call(one, None)))
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("rows,hq,hkv,d,inter,sections", [(2500, 8, 2, 128, False, (16, 24, 24)), (1700, 5, 3, 192, False, (9, 11, 12)),
                                                          (1301, 9, 1, 256, True, (22, 53, 53)), (900, 7, 2, 512, False, (1, 127, 2, 126)),
                                                          (3001, 17, 1, 128, True, (1, 2, 3, 58))])
def test_many_tokens(rows, hq, hkv, d, inter, sections):
    """The rings, several rounds of every warp; bad positions on one axis or another."""
    q, k, qd, kd, wq, wk, table, _ = make(rows, hq, hkv, d, 2 * sum(sections), BF, True)
    pos = axes_positions(rows, len(sections), 3)
    at = torch.tensor([0, 5, rows // 2, rows - 1])
    bad = torch.zeros(rows, dtype=torch.bool)
    bad[at] = True
    p = pos.clone()
    for i, (row, x) in enumerate(zip(at, (-1, MAX, 2 ** 31 - 1, -2 ** 31))):
        p[i % len(sections), row] = x
    # the axes' rows may lie in a longer buffer
    wide = torch.zeros(len(sections), rows + 13, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + rows] = p.cuda()
    qo, ko = (torch.full((rows, h, d), 6.0, device="cuda").bfloat16() for h in (hq, hkv))
    sdpa.sdpa_qk_norm_rope(qd, kd, dev(wq), dev(wk), dev(table), wide[:, 5:5 + rows], eps=EPS, interleaved=inter, q_out=qo,
                           k_out=ko, sections=sections)
    assert sdpa.sdpa_get_device_error() == 10
    assert bool((qo.cpu()[bad] == 6).all()) and bool((ko.cpu()[bad] == 6).all())
    angles, row = merged(table, pos, sections), torch.arange(rows)[~bad]
    check_forward(qo.cpu()[~bad], q[~bad], wq, angles, row, 2 * sum(sections), inter, BF)
    check_forward(ko.cpu()[~bad], k[~bad], wk, angles, row, 2 * sum(sections), inter, BF)
    g = torch.Generator().manual_seed(4)
    gq, gk = torch.randn(q.shape, generator=g).bfloat16(), torch.randn(k.shape, generator=g).bfloat16()
    got = sdpa.sdpa_qk_norm_rope_bwd(dev(gq), dev(gk), qd, kd, dev(wq), dev(wk), dev(table), dev(p), eps=EPS,
                                     interleaved=inter, sections=sections)
    assert sdpa.sdpa_get_device_error() == 10
    for x, w, dy, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        want, mag, want_w, mag_w = ref.norm_rope_bwd(dy[~bad], x[~bad], w, angles[~bad], 2 * sum(sections), EPS, inter)
        within(dx.cpu()[~bad], want, mag, ref.U[BF], ref.TINY[BF], 2.0 ** -17)
        within(dw, want_w, mag_w, 0.0, 0.0, 2.0 ** -15)
        assert not dx.cpu()[bad].any()


def test_batched_layout_and_graph():
    """[batch, sequence] tokens, and a captured call replayed with other positions in place."""
    sections, b, s = (16, 24, 24), 3, 50
    q, k, qd, kd, wq, wk, table, _ = make(b * s, 8, 2, 128, 128, BF, False)
    pos = axes_positions(b * s, 3, 5).cuda()
    args = (dev(wq), dev(wk), dev(table))
    flat = sdpa.sdpa_qk_norm_rope(qd, kd, *args, pos, sections=sections)
    shaped = sdpa.sdpa_qk_norm_rope(qd.view(b, s, 8, 128), kd.view(b, s, 2, 128), *args, pos.view(3, b, s), sections=sections)
    assert torch.equal(flat[0].view(b, s, 8, 128), shaped[0]) and torch.equal(flat[1].view(b, s, 2, 128), shaped[1])
    held, qo, ko = pos.clone(), torch.empty_like(qd), torch.empty_like(kd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdpa.sdpa_qk_norm_rope(qd, kd, *args, held, sections=sections, q_out=qo, k_out=ko)
    held.copy_(pos.flip(0))
    graph.replay()
    want = sdpa.sdpa_qk_norm_rope(qd, kd, *args, pos.flip(0).contiguous(), sections=sections)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


@pytest.mark.parametrize("d,dv,inter,sections", [(128, 128, False, (22, 21, 21)), (192, 128, True, (8, 8)),
                                                 (256, 256, False, (24, 20, 20)), (512, 512, False, (100, 100, 50, 6))])
def test_append(d, dv, inter, sections):
    from test_gpu_paged_append import batch, expected

    s = batch(2, [3, 0, 70, 1], [3, 40, 129, 64], 16, 2, d, dv, "hnd", BF, pad=3, hq=6)
    wq, wk = (1 + 0.2 * torch.randn(2, d, device="cuda")).bfloat16()
    table = ref.angles_table(1000, 2 * sum(sections)).cuda()
    pos = axes_positions(s["k"].shape[0], len(sections), 6, 1000).cuda()
    q_ref, k_ref = sdpa.sdpa_qk_norm_rope(s["q"], s["k"], wq, wk, table, pos, interleaved=inter, sections=sections)
    kc, vc = expected(s, k_ref, s["v"])
    q_out = torch.full_like(q_ref, 5.0)
    sdpa.sdpa_paged_append(s["k"], s["v"], s["kc"], s["vc"], *s["dev"], cache_layout="hnd", q=s["q"], q_weight=wq,
                           k_weight=wk, cos_sin=table, positions=pos, interleaved=inter, sections=sections, q_out=q_out)
    assert torch.equal(s["kc"], kc) and torch.equal(s["vc"], vc)
    assert torch.equal(q_out[:-3], q_ref[:-3]) and bool((q_out[-3:] == 5).all())
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("rows,hq,hkv,d,inter,fused,sections",
                         [c for c in CASES if c[0] < 100] + [(5000, 8, 2, 128, False, True, (22, 21, 21))])
def test_every_access_is_inside_the_buffers(rows, hq, hkv, d, inter, fused, sections):
    """The address-checked build, forward and gradient, positions in rows of a wider tensor: the other build's bits."""
    q, k, qd, kd, wq, wk, table, _ = make(rows, hq, hkv, d, 2 * sum(sections), BF, fused)
    wide = torch.full((len(sections), rows + 5), -1, dtype=torch.int32)
    wide[:, :rows] = axes_positions(rows, len(sections), 8)
    pos = wide.cuda()[:, :rows]
    args = (qd, kd, dev(wq), dev(wk), dev(table))
    kw = dict(eps=EPS, interleaved=inter, sections=sections)
    gq, gk = torch.randn_like(qd).contiguous(), torch.randn_like(kd).contiguous()
    want = sdpa.sdpa_qk_norm_rope(*args, pos, **kw) + sdpa.sdpa_qk_norm_rope_bwd(gq, gk, *args, pos, **kw)
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        got = sdpa.sdpa_qk_norm_rope(*args, pos, **kw) + sdpa.sdpa_qk_norm_rope_bwd(gq, gk, *args, pos, **kw)
        assert sdpa.sdpa_debug_address_report()[0] == 0 and sdpa.sdpa_get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_captured_and_on_two_streams():
    sections, rows = (16, 24, 24), 4000
    q, k, qd, kd, wq, wk, table, _ = make(rows, 8, 2, 128, 128, BF, True)
    args = (qd, kd, dev(wq), dev(wk), dev(table))
    a, b = (axes_positions(rows, 3, seed).cuda() for seed in (9, 10))
    gq, gk = torch.randn_like(qd).contiguous(), torch.randn_like(kd).contiguous()
    want = [sdpa.sdpa_qk_norm_rope_bwd(gq, gk, *args, p, sections=sections) for p in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [sdpa.sdpa_qk_norm_rope_bwd(gq, gk, *args, p, sections=sections, stream=s) for p, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(x, y))
    held, graph = a.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sdpa.sdpa_qk_norm_rope_bwd(gq, gk, *args, held, sections=sections)
    for p, y in ((b, want[1]), (a, want[0])):
        held.copy_(p)
        graph.replay()
        assert all(torch.equal(u, v) for u, v in zip(out, y))
