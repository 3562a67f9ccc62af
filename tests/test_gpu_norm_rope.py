"""Per-head norm + rotation and its gradient against a 64-bit reference.

Tolerances, before the first run. With u half a step of the output's type, the
only 16-bit rounding is the store's: u |y|. In fp32 (2^-24 a rounding): the sum
of D squares is at most 16 products and adds per lane and 5 butterfly steps, 21
roundings, half of which reach r; rsqrtf is within 2 ulp (4 roundings); mean,
two products, and the rotation's two products and one add: below 32 roundings,
2^-19, of the magnitudes |a| + |b| that enter a value. The gradient's dot
product has 21 + 2 roundings, r^3 three times r's 15, and some ten products:
below 128, 2^-17, of its magnitudes. dw adds at most 256 terms in a row per
lane, block and column for the sizes here (rows x heads <= 12000, spread over
hundreds of lanes): (256 + 64) 2^-24 < 2^-15 of the summed magnitudes.
"""
import numpy as np
import pytest
import torch

import paged_ref as ref
import scaled_dot_product_02_gb300 as sdpa

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(rows, hq, hkv, d, rot, dtype, fused, seed=0, max_pos=5000):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if fused:
        whole = n(rows, (hq + 2 * hkv) * d).to(dtype)
        q = whole[:, :hq * d].unflatten(1, (hq, d))
        k = whole[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        dev = whole.cuda()
        qd = dev[:, :hq * d].unflatten(1, (hq, d))
        kd = dev[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    else:
        q, k = n(rows, hq, d).to(dtype), n(rows, hkv, d).to(dtype)
        qd, kd = q.cuda(), k.cuda()
    wq, wk = (1 + 0.3 * n(d)).to(dtype), (1 + 0.3 * n(d)).to(dtype)
    table = ref.angles_table(max_pos, rot)
    pos = torch.from_numpy(np.random.default_rng(seed).integers(0, max_pos, rows).astype(np.int32))
    return q, k, qd, kd, wq, wk, table, pos


def dev(t):
    return None if t is None else t.cuda()


def within(got, want, mag, u, tiny, slack):
    err = (got.double().cpu() - want).abs()
    tol = u * want.abs() + tiny + slack * mag
    assert bool((err <= tol).all()), f"worst {(err / tol.clamp(min=1e-300)).max().item():.3f} of the tolerance"


def check_forward(out, x, w, table, pos, rot, inter, dtype, eps=EPS):
    rows = None if rot == 0 else table[pos.long()]
    want, mag = ref.norm_rope(x, w, rows, rot, eps, inter)
    within(out, want, mag, ref.U[dtype], ref.TINY[dtype], 2.0 ** -19)


CASES = [(1, 32, 8, 128, 128, False, True), (77, 32, 8, 128, 128, True, False), (5, 3, 1, 128, 16, False, False),
         (300, 16, 4, 128, 64, False, True), (19, 14, 2, 192, 192, False, True), (33, 4, 4, 192, 96, True, False),
         (21, 16, 8, 256, 256, False, False), (64, 16, 8, 256, 128, True, True), (9, 2, 2, 256, 0, False, False),
         (13, 16, 4, 512, 512, False, True), (40, 5, 5, 512, 208, False, False), (2, 1, 1, 512, 512, True, False)]


@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter,fused", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forward(rows, hq, hkv, d, rot, inter, fused, dtype):
    q, k, qd, kd, wq, wk, table, pos = make(rows, hq, hkv, d, rot, dtype, fused)
    qo, ko = sdpa.sdpa_qk_norm_rope(qd, kd, dev(wq), dev(wk), dev(table), dev(pos) if rot else None, eps=EPS,
                                    interleaved=inter)
    assert sdpa.sdpa_last_launch_count() == 1
    check_forward(qo, q, wq, table, pos, rot, inter, dtype)
    check_forward(ko, k, wk, table, pos, rot, inter, dtype)
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter,fused", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_backward(rows, hq, hkv, d, rot, inter, fused, dtype):
    q, k, qd, kd, wq, wk, table, pos = make(rows, hq, hkv, d, rot, dtype, fused)
    g = torch.Generator().manual_seed(9)
    gq, gk = torch.randn(q.shape, generator=g).to(dtype), torch.randn(k.shape, generator=g).to(dtype)
    args = (dev(gq), dev(gk), qd, kd, dev(wq), dev(wk), dev(table), dev(pos) if rot else None)
    got = sdpa.sdpa_qk_norm_rope_bwd(*args, eps=EPS, interleaved=inter)
    rows_t = None if rot == 0 else table[pos.long()]
    for x, w, dy, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        want, mag, want_w, mag_w = ref.norm_rope_bwd(dy, x, w, rows_t, rot, EPS, inter)
        within(dx, want, mag, ref.U[dtype], ref.TINY[dtype], 2.0 ** -17)
        within(dw, want_w, mag_w, 0.0, 0.0, 2.0 ** -15)
    again = sdpa.sdpa_qk_norm_rope_bwd(*args, eps=EPS, interleaved=inter)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # the gradient written into slices of one fused gradient's rows
    fused_g = torch.zeros(rows, (hq + 2 * hkv) * d, dtype=dtype, device="cuda")
    dq = fused_g[:, :hq * d].unflatten(1, (hq, d))
    dk = fused_g[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    sdpa.sdpa_qk_norm_rope_bwd(*args, eps=EPS, interleaved=inter, dq=dq, dk=dk)
    assert torch.equal(dq, got[0]) and torch.equal(dk, got[1])
    assert not fused_g[:, (hq + hkv) * d:].any()
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter", [(2500, 8, 2, 128, 128, False), (1700, 5, 3, 192, 64, False),
                                                     (1301, 9, 1, 256, 256, True), (900, 7, 2, 512, 512, False),
                                                     (3001, 17, 1, 128, 0, False)])
def test_many_tokens(rows, hq, hkv, d, rot, inter):
    """Enough units for every warp of the rings to go round several times; a few positions are bad."""
    q, k, qd, kd, wq, wk, table, pos = make(rows, hq, hkv, d, rot, torch.bfloat16, True)
    bad = torch.zeros(rows, dtype=torch.bool)
    p = pos.clone()
    if rot:
        bad[torch.tensor([0, 5, rows // 2, rows - 1])] = True
        p[bad] = torch.tensor([-1, 5000, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    qo, ko = torch.full((rows, hq, d), 6.0, device="cuda").bfloat16(), torch.full((rows, hkv, d), 6.0, device="cuda").bfloat16()
    sdpa.sdpa_qk_norm_rope(qd, kd, dev(wq), dev(wk), dev(table), dev(p) if rot else None, eps=EPS, interleaved=inter,
                           q_out=qo, k_out=ko)
    assert sdpa.sdpa_get_device_error() == (10 if rot else 0)
    assert bool((qo.cpu()[bad] == 6).all()) and bool((ko.cpu()[bad] == 6).all())
    check_forward(qo.cpu()[~bad], q[~bad], wq, table, pos[~bad], rot, inter, torch.bfloat16)
    check_forward(ko.cpu()[~bad], k[~bad], wk, table, pos[~bad], rot, inter, torch.bfloat16)
    g = torch.Generator().manual_seed(4)
    gq, gk = torch.randn(q.shape, generator=g).bfloat16(), torch.randn(k.shape, generator=g).bfloat16()
    args = (dev(gq), dev(gk), qd, kd, dev(wq), dev(wk), dev(table), dev(p) if rot else None)
    got = sdpa.sdpa_qk_norm_rope_bwd(*args, eps=EPS, interleaved=inter)
    again = sdpa.sdpa_qk_norm_rope_bwd(*args, eps=EPS, interleaved=inter)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert sdpa.sdpa_get_device_error() == (10 if rot else 0)
    keep = ~bad
    rows_t = None if rot == 0 else table[pos[keep].long()]
    for x, w, dy, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        want, mag, want_w, mag_w = ref.norm_rope_bwd(dy[keep], x[keep], w, rows_t, rot, EPS, inter)
        within(dx.cpu()[keep], want, mag, ref.U[torch.bfloat16], 0.0, 2.0 ** -17)
        within(dw, want_w, mag_w, 0.0, 0.0, 2.0 ** -15)
        assert not dx.cpu()[bad].any()


@pytest.mark.parametrize("layout", ["bshd", "sbhd"])
def test_batched_layouts(layout):
    a, b = (3, 41) if layout == "bshd" else (41, 3)
    q, k, qd, kd, wq, wk, table, pos = make(a * b, 4, 2, 128, 128, torch.bfloat16, False)
    qo, ko = sdpa.sdpa_qk_norm_rope(qd.view(a, b, 4, 128), kd.view(a, b, 2, 128), dev(wq), dev(wk), dev(table),
                                    dev(pos).view(a, b), eps=EPS)
    assert qo.shape == (a, b, 4, 128) and ko.shape == (a, b, 2, 128)
    check_forward(qo.view(a * b, 4, 128), q, wq, table, pos, 128, False, torch.bfloat16)
    check_forward(ko.view(a * b, 2, 128), k, wk, table, pos, 128, False, torch.bfloat16)


def test_zero_rows_and_special_values_stay_in_their_rows():
    q, k, qd, kd, wq, wk, table, pos = make(8, 4, 2, 128, 128, torch.bfloat16, False)
    qd = qd.clone()
    qd[2, 1] = 0.0
    qd[3, 0, 5] = float("nan")
    qd[4, 3, 100] = float("inf")
    args = (dev(wq), dev(wk), dev(table), dev(pos))
    qo, _ = sdpa.sdpa_qk_norm_rope(qd, kd, *args, eps=EPS)
    assert not qo[2, 1].any()
    bad = ~torch.isfinite(qo).all(-1)
    assert bad.nonzero().tolist() == [[3, 0], [4, 3]]
    keep = ~bad.cpu()
    want, mag = ref.norm_rope(qd.cpu(), wq, table[pos.long()], 128, EPS, False)
    within(qo.cpu()[keep], want[keep], mag[keep], ref.U[torch.bfloat16], 0.0, 2.0 ** -19)


def test_bad_positions_are_recorded_and_their_rows_left():
    q, k, qd, kd, wq, wk, table, pos = make(9, 4, 2, 128, 64, torch.bfloat16, False, max_pos=100)
    bad = dev(pos).clone()
    bad[4], bad[7] = 100, -1
    qo, ko = torch.full_like(qd, 7.0), torch.full_like(kd, 7.0)
    sdpa.sdpa_qk_norm_rope(qd, kd, dev(wq), dev(wk), dev(table), bad, eps=EPS, q_out=qo, k_out=ko)
    assert sdpa.sdpa_get_device_error() == 10
    live = torch.tensor([i not in (4, 7) for i in range(9)])
    assert bool((qo.cpu()[~live] == 7).all()) and bool((ko.cpu()[~live] == 7).all())
    check_forward(qo.cpu()[live], q[live], wq, table, pos[live], 64, False, torch.bfloat16)
    gq, gk = torch.randn_like(qd), torch.randn_like(kd)
    dq, dk, dwq, dwk = sdpa.sdpa_qk_norm_rope_bwd(gq, gk, qd, kd, dev(wq), dev(wk), dev(table), bad, eps=0.0)
    assert sdpa.sdpa_get_device_error() == 10
    assert not dq.cpu()[~live].any() and not dk.cpu()[~live].any()
    want = sdpa.sdpa_qk_norm_rope_bwd(gq[live.cuda()], gk[live.cuda()], qd[live.cuda()], kd[live.cuda()], dev(wq), dev(wk),
                                      dev(table), bad[live.cuda()], eps=0.0)
    assert torch.equal(dq[live.cuda()], want[0]) and torch.equal(dk[live.cuda()], want[1])
    assert sdpa.sdpa_get_device_error() == 0


def test_no_rows():
    _, _, _, _, wq, wk, table, _ = make(1, 4, 2, 128, 64, torch.bfloat16, False)
    z = lambda h: torch.zeros(0, h, 128, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    qo, ko = sdpa.sdpa_qk_norm_rope(z(4), z(2), dev(wq), dev(wk), dev(table), pos)
    assert qo.shape == (0, 4, 128) and ko.shape == (0, 2, 128)
    dwq = torch.full((128,), 3.0, device="cuda")
    got = sdpa.sdpa_qk_norm_rope_bwd(z(4), z(2), z(4), z(2), dev(wq), dev(wk), dev(table), pos, dq_weight=dwq)
    assert not dwq.any() and not got[3].any()


def test_captured_and_on_another_stream():
    q, k, qd, kd, wq, wk, table, pos = make(50, 8, 2, 128, 128, torch.bfloat16, True)
    args = (dev(wq), dev(wk), dev(table))
    p = dev(pos)
    gq, gk = torch.randn(50, 8, 128, device="cuda").bfloat16(), torch.randn(50, 2, 128, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = sdpa.sdpa_qk_norm_rope(qd, kd, *args, p, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = sdpa.sdpa_qk_norm_rope(qd, kd, *args, p)
        c = sdpa.sdpa_qk_norm_rope_bwd(gq, gk, qd, kd, *args, p)
    for turn in range(2):
        p.copy_((dev(pos) + turn) % 5000)
        graph.replay()
        want = sdpa.sdpa_qk_norm_rope(qd, kd, *args, p)
        back = sdpa.sdpa_qk_norm_rope_bwd(gq, gk, qd, kd, *args, p)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(b, want))
        assert all(torch.equal(x, y) for x, y in zip(c, back))
        if turn == 0:
            assert all(torch.equal(x, y) for x, y in zip(a, want))


@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (192, 96, True), (256, 64, False), (512, 512, False)])
@pytest.mark.parametrize("n", [37, 2600])
def test_every_access_is_inside_the_buffers(d, rot, inter, n):
    q, k, qd, kd, wq, wk, table, pos = make(n, 6, 2, d, rot, torch.float16, True)
    args = (dev(wq), dev(wk), dev(table), dev(pos))
    gq, gk = torch.randn(n, 6, d, device="cuda").half(), torch.randn(n, 2, d, device="cuda").half()
    plain = sdpa.sdpa_qk_norm_rope(qd, kd, *args, interleaved=inter) + sdpa.sdpa_qk_norm_rope_bwd(
        gq, gk, qd, kd, *args, interleaved=inter)
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        got = sdpa.sdpa_qk_norm_rope(qd, kd, *args, interleaved=inter) + sdpa.sdpa_qk_norm_rope_bwd(
            gq, gk, qd, kd, *args, interleaved=inter)
        assert sdpa.sdpa_debug_address_report()[0] == 0
    assert all(torch.equal(a, b) for a, b in zip(plain, got))


@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 64, True), (192, 192, False), (256, 128, True), (512, 512, False)])
@pytest.mark.parametrize("scale,eps", [(1e15, EPS), (1e17, EPS), (1e-13, 0.0), (1e-18, 0.0)])
def test_gradient_of_rows_far_from_unit_scale(d, rot, inter, scale, eps):
    """dx is some 1 / scale and dw does not depend on it, though r^3 alone leaves the range of fp32."""
    q, k, _, _, wq, wk, table, pos = make(60, 6, 2, d, rot, torch.bfloat16, False)
    q, k = (q.float() * scale).bfloat16(), (k.float() * scale).bfloat16()
    g = torch.Generator().manual_seed(9)
    gq, gk = torch.randn(q.shape, generator=g).bfloat16(), torch.randn(k.shape, generator=g).bfloat16()
    got = sdpa.sdpa_qk_norm_rope_bwd(dev(gq), dev(gk), dev(q), dev(k), dev(wq), dev(wk), dev(table), dev(pos), eps=eps,
                                     interleaved=inter)
    for x, w, dy, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        want, mag, want_w, mag_w = ref.norm_rope_bwd(dy, x, w, table[pos.long()], rot, eps, inter)
        within(dx, want, mag, ref.U[torch.bfloat16], 0.0, 2.0 ** -17)
        within(dw, want_w, mag_w, 0.0, 0.0, 2.0 ** -15)
    assert sdpa.sdpa_get_device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 64), (192, 96), (256, 64), (512, 16)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_weight_that_is_not_finite_stays_in_its_column(inter, d, rot, value):
    """Where nothing turns the result is x r w alone, for few tokens and for many; a pair takes the weight in both halves."""
    q, k, qd, kd, wq, wk, table, pos = make(3800, 4, 1, d, rot, torch.bfloat16, True)
    table[:, rot // 2:] = table[:, rot // 2:].abs().clamp(min=0.1)  # a sine of zero times an infinity would be NaN
    tail, pair = d - 3, 2                                           # an unrotated column, a rotated one
    for at in (tail, pair):
        w = wq.clone()
        w[at] = value
        hit = {at} if at == tail else {at, ref.pair_index(d, rot, inter)[0][at].item()}
        keep = torch.tensor([i not in hit for i in range(d)])
        for n in (3, 3800):
            qo, ko = sdpa.sdpa_qk_norm_rope(qd[:n], kd[:n], dev(w), dev(w), dev(table), dev(pos[:n]), eps=EPS, interleaved=inter)
            for out, x in ((qo.cpu(), q[:n]), (ko.cpu(), k[:n])):
                want, mag = ref.norm_rope(x, w, table[pos[:n].long()], rot, EPS, inter)
                within(out[..., keep], want[..., keep], mag[..., keep], ref.U[torch.bfloat16], 0.0, 2.0 ** -19)
                for i in hit:  # x or its partner may be zero: NaN then, as in the definition
                    assert torch.equal(out[..., i].float().nan_to_num(9.0, 2.0, -2.0),
                                       want[..., i].float().nan_to_num(9.0, 2.0, -2.0))


@pytest.mark.parametrize("hq,hkv,d,rot,inter,dtype,fused", [
    (8, 2, 128, 128, False, torch.bfloat16, True), (17, 1, 128, 64, True, torch.float16, False),
    (16, 4, 128, 32, False, torch.float16, True), (11, 3, 192, 192, False, torch.float16, True),
    (4, 4, 192, 96, True, torch.bfloat16, False), (9, 1, 256, 256, True, torch.bfloat16, True),
    (8, 2, 256, 64, False, torch.float16, False), (16, 16, 256, 192, False, torch.bfloat16, False),
    (7, 2, 512, 512, False, torch.bfloat16, True), (4, 1, 512, 208, True, torch.float16, False),
    (3, 2, 512, 16, False, torch.bfloat16, True)])
def test_the_rings_of_many_tokens(hq, hkv, d, rot, inter, dtype, fused):
    """At least three units for every one of the 24 warps of each SM (a unit is 4 KB of one tensor's heads of a token), with
    one and two stages a warp; bad positions, in a row for one warp too, and infinities beside pairs and in them."""
    per = 4096 // (2 * d)
    parts = -(-hq // per) - (-hkv // per)
    warps = 24 * torch.cuda.get_device_properties(0).multi_processor_count
    rows = -(-3 * warps // parts) + 5
    q, k, qd, kd, wq, wk, table, pos = make(rows, hq, hkv, d, rot, dtype, fused, seed=d + rot)
    for row, head, col in ((3, 0, d - 1), (4, hq - 1, 1), (rows - 2, 0, rot - 1), (rows // 2, hq // 2, rot % d)):
        q[row, head, col] = qd[row, head, col] = float("inf")
    bad = torch.zeros(rows, dtype=torch.bool)
    bad[[0, 7, rows - 1] + [11 + i * warps // parts for i in range(3)]] = True  # the last three: one warp's first units
    p = pos.clone()
    p[bad] = torch.tensor([-1, 5000, 2 ** 31 - 1, -2 ** 31, 6000, -7], dtype=torch.int32)
    qo = torch.full((rows, hq, d), 6.0, dtype=dtype, device="cuda")
    ko = torch.full((rows, hkv, d), 6.0, dtype=dtype, device="cuda")
    args = (qd, kd, dev(wq), dev(wk), dev(table), dev(p))
    sdpa.sdpa_qk_norm_rope(*args, eps=EPS, interleaved=inter, q_out=qo, k_out=ko)
    assert sdpa.sdpa_get_device_error() == 10
    assert bool((qo.cpu()[bad] == 6).all()) and bool((ko.cpu()[bad] == 6).all())
    for out, x, w in ((qo, q, wq), (ko, k, wk)):
        out = out.cpu()[~bad]
        want, mag = ref.norm_rope(x[~bad], w, table[pos[~bad].long()], rot, EPS, inter)
        finite = torch.isfinite(want)
        assert torch.equal(torch.isfinite(out), finite)
        within(out[finite], want[finite], mag[finite], ref.U[dtype], ref.TINY[dtype], 2.0 ** -19)
    with sdpa.address_checked():
        sdpa.sdpa_debug_address_report()
        again = sdpa.sdpa_qk_norm_rope(*args, eps=EPS, interleaved=inter)
        assert sdpa.sdpa_debug_address_report()[0] == 0
        assert sdpa.sdpa_get_device_error() == 10
    good = (~bad).cuda()
    for a, b in zip(again, (qo, ko)):
        assert torch.equal(a[good].view(torch.int16), b[good].view(torch.int16))
